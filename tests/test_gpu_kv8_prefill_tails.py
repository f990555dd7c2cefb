"""gqa_kv8_prefill where one key takes nearly all probability and very many others share the rest: what they say
together comes out as the formula has it, as in gqa_kv8_decode."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, f8, i32
from tests.parity import to_f64
from tests.test_gpu_kv8_tails import GAPS, U, _case, _reference

pytestmark = pytest.mark.gpu


def _run(kp, vp, bs, n, q, B, rows, dtype):
    """B sequences that share one table of n keys, each with `rows` rows of the same q [8, 256]."""
    T = B * rows
    qd = q.to(dtype).to(DEV).expand(T, 8, 256).contiguous()
    ones = torch.ones(kp.shape[0], 1, device=DEV)
    tables = torch.arange(kp.shape[0], dtype=torch.int32, device=DEV).expand(B, -1).contiguous()
    cu = torch.arange(0, T + 1, rows, dtype=torch.int32, device=DEV)
    out = G.kv8_prefill(qd, kp, vp, ones, ones * 2.0**-6, None, tables, i32([n] * B), cu, max_rows=rows, max_kv_len=n)
    assert G.last_device_status() == 0
    return to_f64(out).reshape(B, rows, 8, 256)


# 160 sequences: every pair has more than two of them, so that pieces are long; one: 76 pairs share it
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,rows", [(160, 8), (1, 40)])
@pytest.mark.parametrize("sink,spread", [(0, False), (70001, False), (0, True), (70001, True)])
def test_many_keys_far_below_one(sink, spread, B, rows, dtype):
    """131071 keys, one of them 11 to 18 nats above the others.

    Tolerance: a probability is off by 2^-11 of itself, sums and scores by 2^-13, the output by half a step u of its
    type.  Beside that a key loses 2^-33 of the one's weight at most where a pair has more than 8192 keys of the row at
    a time, and else 2^-25 or its own weight again, whichever is less: together 131071 * 2^-33 + 8192 * 2^-25 of the
    one's, which is below that of all, and the values are 1.25 at most.  Of the keys' own weight, 18 nats below on
    average or nearer (2^-25.97), 2^-33 is 2^-7; and the 8192 keys of one short piece are 64 / 1024 of it (70 where
    weights are spread: 8192 of them, of variance e - 1, are within 6 % of their mean)."""
    n, bs = 131071, 128
    k, v, kp, vp = _case(n, bs, sink, spread, 220)
    q = torch.zeros(8, 256)
    q[:, 0] = torch.tensor(GAPS) / 8.0
    q[:, 1] = float(spread)
    got = _run(kp, vp, bs, n, q, B, rows, dtype)
    for i in {0, rows - 1}:
        ref = _reference(k, v, n - rows + i + 1, q[:, :2].double().numpy())
        err = np.abs(got[:, i] - ref[None])
        rel = U[dtype] + 2.0**-11 + 2.0**-13
        assert np.all(err <= rel * ref[None] + 1.25 * (2.0**-16 + 2.0**-12))
        assert np.all(err.max((0, 2)) <= ref.max(1) * (rel + 2.0**-7 + 70 / 1024))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("per", [3, 12])
def test_a_staircase_of_keys(per, dtype):
    """Tiles that go up and down by tens of nats, past what one reference holds, and down to what no sum can see, in
    pieces of at most 64 tiles and of more."""
    bs, B, rows = 64, 160, 8
    n = 128 * 20 * per
    gen = torch.Generator().manual_seed(221)
    heights = torch.tensor([0, 40, 12, 39, -60, 5, 41, 20, 41.5, -100, 38, 41, 0, 30, 10, 40.5, 41, 42, 7, 42])
    k = np.zeros((n, 256), dtype=np.uint8)
    k[:, 0] = oracle.e4m3_encode((heights.repeat_interleave(per * 128) * 4).double().numpy())   # q 4: k / 16 * 4 nats
    k[:, 1] = oracle.e4m3_encode((torch.randn(n, generator=gen) * 16).double().numpy())
    v = oracle.e4m3_encode((torch.randn(n, 256, generator=gen) * 64).double().numpy())
    q = torch.zeros(8, 256)
    q[:, 0] = torch.tensor([4.0, 2, 1, 0.5, -4, -1, 3, 0.25])
    q[:, 1] = 1.0
    shape = (n // bs, 1, bs, 256)
    got = _run(f8(k.reshape(shape)), f8(v.reshape(shape)), bs, n, q, B, rows, dtype)
    # |V| <= 7: sums of weighted |V| are below it.  Probabilities 2^-11 of themselves, the output u of itself; scores
    # reach 450 / 4 with fp32 errors of 2^-24 of it and sums 2^-13; a segment is cut once at most, and what a row's
    # keys lose together is 2^-12 (8192 of a short piece, 2^-25 each) and 2^-18 (30720 of a long one).
    tol = 7 * (U[dtype] + 2.0**-11 + 2.0**-13 + 2.0**-12 + 2.0**-18)
    for i in (0, rows - 1):
        ref = _reference(k, v, n - rows + i + 1, q[:, :2].double().numpy())
        assert np.abs(got[:, i] - ref[None]).max() <= tol
