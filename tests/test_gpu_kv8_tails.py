"""One key that takes nearly all probability, and very many others that share the rest: what they say
together has to come out as the formula has it, however far below the one they are."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, f8, i32
from tests.parity import to_f64

pytestmark = pytest.mark.gpu

GAPS = [11, 12, 13, 14, 15, 16, 17, 18]         # nats of the one key above the others, a head each
U = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def _case(n, bs, sink, spread, seed):
    """A sequence of n keys in order in one pool: K is 0 but for dim 0 of the sink (128) and, where
    `spread`, dim 1 (16 N(0, 1): one nat of standard deviation); V about 1, 0 for the sink."""
    gen = torch.Generator().manual_seed(seed)
    blocks = -(-n // bs)
    rows = blocks * bs
    k = np.zeros((rows, 256), dtype=np.uint8)
    if spread:
        k[:, 1] = oracle.e4m3_encode((torch.randn(rows, generator=gen) * 16).double().numpy())
        k[sink, 1] = 0
    k[sink, 0] = int(oracle.e4m3_encode(np.array([128.0]))[0])
    v = oracle.e4m3_encode((48 + 32 * torch.rand(rows, 256, generator=gen)).double().numpy())
    v[sink] = 0
    shape = (blocks, 1, bs, 256)
    return k, v, f8(k.reshape(shape)), f8(v.reshape(shape))


def _reference(k, v, n, q):
    """[heads, 256] in float64, values of V by 2^-6."""
    s = np.stack([oracle.E4M3[k[:n, 0]], oracle.E4M3[k[:n, 1]]], 1) @ q.T / 16
    w = np.exp(s - s.max(0))
    return (w / w.sum(0)).T @ (oracle.E4M3[v[:n]] * 2.0**-6)


# 8 heads x 1, 3, 4 rows: the kernel for few rows; x 8: the one for many
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 3, 4, 8])
@pytest.mark.parametrize("sink,spread", [(0, False), (70001, False), (0, True), (70001, True), (131070 - 8, False)])
def test_many_keys_far_below_one(sink, spread, rows, dtype):
    """131071 keys, read by so many sequences that no CTA has much less than one to itself.

    Tolerance: a probability's terms are off by half a step of the output's type at most (the kernel
    for many rows; 2^-13 the other), the output's rounding by another, sums and scores by 2^-13; so
    3 u of the value.  The keys of the tiles that the one key's own reference holds for, 17 at most,
    lose 2^-24 of its weight each: 17 * 128 * 2^-24 < 2^-12 of the largest V, 1.25, over the weight
    of all (1 and more); so with the 65 tiles at 2^-25 of a share of at most 64 (2^-24 for many rows,
    where 64 * 128 * 2^-24 = 2^-11 is the bound)."""
    n, bs, B = 131071, 128, 160
    k, v, kp, vp = _case(n, bs, sink, spread, 150)
    q = torch.zeros(8, 256)
    q[:, 0] = torch.tensor(GAPS) / 8.0
    q[:, 1] = float(spread)
    ref = _reference(k, v, n, q[:, :2].double().numpy())
    T = B * rows
    qd = q.to(dtype).to(DEV).expand(T, 8, 256).contiguous()
    ones = torch.ones(kp.shape[0], 1, device=DEV)
    tables = torch.arange(kp.shape[0], dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    cu = torch.arange(0, T + 1, rows, dtype=torch.int32, device=DEV)
    mask = torch.full((T,), (1 << rows) - 1, dtype=torch.int64, device=DEV)    # every row sees all keys
    out = G.kv8_decode(qd, kp, vp, ones, ones * 2.0**-6, None, tables, i32([n] * B), cu, tree_mask=mask,
                       max_rows=rows, max_kv_len=n)
    assert G.last_device_status() == 0
    err = np.abs(to_f64(out) - ref[None])
    tol = 3 * U[dtype] * ref + 2.0**-12 * 1.25
    # and of a row's own value no more than 65 of its 1024 tiles are worth: those of a CTA's share of
    # at most 64, in which references stay where they are, and the one of the one key
    assert np.all(err <= tol[None])
    assert np.all(err.max((0, 2)) <= ref.max(1) * (3 * U[dtype] + 65 / 1024))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 8])
def test_a_staircase_of_keys(rows, dtype):
    """Tiles that go up and down by tens of nats, past what one reference holds, and down to what no sum
    can see: the values stay finite and right."""
    n, bs = 128 * 60, 64
    gen = torch.Generator().manual_seed(151)
    heights = torch.tensor([0, 40, 12, 39, -60, 5, 41, 20, 41.5, -100, 38, 41, 0, 30, 10, 40.5, 41, 42, 7, 42])
    k = np.zeros((n, 256), dtype=np.uint8)
    per = heights.repeat_interleave(3 * 128)
    k[:, 0] = oracle.e4m3_encode((per * 4).double().numpy())           # q 4: k / 16 * 4 nats
    k[:, 1] = oracle.e4m3_encode((torch.randn(n, generator=gen) * 16).double().numpy())
    v = oracle.e4m3_encode((torch.randn(n, 256, generator=gen) * 64).double().numpy())
    q = torch.zeros(8, 256)
    q[:, 0] = torch.tensor([4.0, 2, 1, 0.5, -4, -1, 3, 0.25])
    q[:, 1] = 1.0
    ref = _reference(k, v, n, q[:, :2].double().numpy())
    B = 160
    T = B * rows
    qd = q.to(dtype).to(DEV).expand(T, 8, 256).contiguous()
    ones = torch.ones(n // bs, 1, device=DEV)
    tables = torch.arange(n // bs, dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    mask = torch.full((T,), (1 << rows) - 1, dtype=torch.int64, device=DEV)
    shape = (n // bs, 1, bs, 256)
    out = G.kv8_decode(qd, f8(k.reshape(shape)), f8(v.reshape(shape)), ones, ones * 2.0**-6, None, tables,
                       i32([n] * B), torch.arange(0, T + 1, rows, dtype=torch.int32, device=DEV),
                       tree_mask=mask, max_rows=rows, max_kv_len=n)
    assert G.last_device_status() == 0
    # |V| <= 7: sums of weighted |V| are below it.  Terms and rounding u each; scores reach 450 / 4 with
    # fp32 errors of 2^-24 of it, 2^-17; the lost parts as above.
    assert np.abs(to_f64(out) - ref[None]).max() <= 7 * (2 * U[dtype] + 2.0**-12)
