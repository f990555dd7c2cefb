"""Rotary positions against float64: layouts, strides, far positions, in place, back again.

An output is (x1 c - x2 s) with c, s off by 2^-23 (the angle to 2^-29 of a radian, sincospif, a float angle of up to
one half turn: 2^-24 pi) and three fp32 roundings: 4 * 2^-23 of |x1| + |x2| at most, scale included, and half a step
of the type of itself (fp16 below 2^-14: 2^-25)."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, i32
from tests.parity import to_f64

pytestmark = pytest.mark.gpu


def _freq(rot, base=10000.0):
    f, scale = G.rope_frequencies(rot, base)
    assert scale == 1.0
    return f


def _bound(x, rot, interleaved, scale, ref, dtype):
    a = np.abs(x) * abs(scale)
    half, pair = rot // 2, np.zeros_like(a)
    i1, i2 = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(half), np.arange(half, rot))
    pair[..., i1] = pair[..., i2] = a[..., i1] + a[..., i2]
    return 4 * 2.0 ** -23 * pair + np.abs(ref) * torch.finfo(dtype).eps / 2 * 1.001 + 2.0 ** -25


def _check(got, x, positions, freq, interleaved=False, scale=1.0, inverse=False):
    xs, rot = to_f64(x), 2 * freq.numel()
    ref = oracle.rope(xs, positions, to_f64(freq), interleaved, scale, inverse)
    err = np.abs(to_f64(got) - ref)
    assert (err <= _bound(xs, rot, interleaved, scale, ref, x.dtype)).all(), err.max()
    assert np.array_equal(to_f64(got)[..., rot:], xs[..., rot:])


def _x(shape, seed, dtype):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(DEV, dtype)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,Hq,Hkv,rot", [(1, 1, 1, 16), (5, 24, 4, 64), (37, 16, 2, 256), (9, 7, 3, 48),
                                          (3, 40, 1, 128), (130, 3, 9, 240)])
def test_token_major(T, Hq, Hkv, rot, dtype, interleaved):
    q, k = _x((T, Hq, 256), 1, dtype), _x((T, Hkv, 256), 2, dtype)
    pos = np.random.RandomState(3).randint(0, 5000, T).tolist()
    f = _freq(rot)
    q2, k2 = G.rope(q, k, i32(pos), f, interleaved=interleaved, scale=1.25)
    assert G.last_device_status() == 0
    _check(q2, q, pos, f, interleaved, 1.25)
    _check(k2, k, pos, f, interleaved, 1.25)


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_and_negative_positions(interleaved):
    pos = [0, 1, -1, 123456789, 2 ** 31 - 1, -2 ** 31, 1000003, 16777217]
    q = _x((len(pos), 2, 256), 4, torch.float16)
    f = _freq(128, 1e6)
    got, none = G.rope(q, None, i32(pos), f, interleaved=interleaved)
    assert none is None
    _check(got, q, pos, f, interleaved)


def test_frequencies_of_any_size():
    f = torch.tensor([0.0, -0.5, 3.0, 1e-30, 1e-42, 250.0, 1.0, 2.0 ** -20], device=DEV)
    q = _x((6, 2, 256), 5, torch.float16)
    pos = [1, 7, 100, 5000, 65535, 3]
    got, _ = G.rope(q, None, i32(pos), f)
    _check(got, q, pos, f)
    f[3] = float("inf")
    got, _ = G.rope(q, None, i32(pos), f)
    bad = torch.isnan(got)
    assert bad[:, :, 3].all() and bad[:, :, 11].all() and bad.sum().item() == 2 * 6 * 2


@pytest.mark.parametrize("batched", [False, True])
def test_prefill_layout(batched):
    B, Hq, Hkv, L, rot = 3, 6, 2, 19, 64
    q, k = _x((B, Hq, L, 256), 6, torch.bfloat16), _x((B, Hkv, L, 256), 7, torch.bfloat16)
    pos = np.random.RandomState(8).randint(0, 9000, (B, L) if batched else L)
    f = _freq(rot)
    q2, k2 = G.rope(q, k, i32(pos.tolist()), f)
    assert q2.is_contiguous() and q2.shape == q.shape
    for b in range(B):
        at = (pos[b] if batched else pos).tolist()
        _check(q2[b].transpose(0, 1), q[b].transpose(0, 1), at, f)
        _check(k2[b].transpose(0, 1), k[b].transpose(0, 1), at, f)


def test_slices_of_a_fused_projection_and_transposed_views():
    T, Hq, Hkv, f = 33, 6, 2, _freq(64)
    x = _x((T, Hq + 2 * Hkv, 256), 9, torch.bfloat16)
    keep = x.clone()
    pos = list(range(100, 100 + T))
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    q2, k2 = G.rope(q, k, i32(pos), f)
    _check(q2, q, pos, f)
    _check(k2, k, pos, f)
    assert torch.equal(x, keep) and q2.is_contiguous()
    # in place, the rest of the projection as it was
    G.rope(q, k, i32(pos), f, q_out=q, k_out=k)
    assert torch.equal(x[:, :Hq], q2) and torch.equal(x[:, Hq:Hq + Hkv], k2)
    assert torch.equal(x[:, Hq + Hkv:], keep[:, Hq + Hkv:])
    # [B, H, L, 256] that is a view of token-major rows, and an output in that view
    y = keep[:, :Hq].contiguous().view(3, 11, Hq, 256)
    out = torch.zeros_like(y)
    G.rope(y.transpose(1, 2), None, i32(np.reshape(pos, (3, 11)).tolist()), f, q_out=out.transpose(1, 2))
    assert torch.equal(out.view(T, Hq, 256), q2)
    # one token's rows for all
    one = _x((1, 4, 256), 10, torch.float16)
    many, _ = G.rope(one.expand(T, 4, 256), None, i32(pos), f)
    _check(many, one.expand(T, 4, 256).cpu(), pos, f)


@pytest.mark.parametrize("interleaved", [False, True])
def test_back_is_the_gradient(interleaved):
    """<rope(x), y> = <x, rope back(y)>: the rotation back is the transposed one, against the formula and
    differences (rope is linear: a difference is the map itself)."""
    T, H, rot, scale = 11, 3, 64, 1.5
    f, pos = _freq(rot), list(range(7, 7 + T))
    y = _x((T, H, 256), 12, torch.float16)
    gx, _ = G.rope(y, None, i32(pos), f, interleaved=interleaved, scale=scale, inverse=True)
    _check(gx, y, pos, f, interleaved, scale, True)
    rng = np.random.RandomState(13)
    for _ in range(20):
        t, h, i = rng.randint(T), rng.randint(H), rng.randint(256)
        e = torch.zeros(T, H, 256, dtype=torch.float16, device=DEV)
        e[t, h, i] = 1.0
        r, _ = G.rope(e, None, i32(pos), f, interleaved=interleaved, scale=scale)
        d = float((to_f64(r) * to_f64(y)).sum())
        # two outputs of r and one of gx, each half a step (2^-11) of scale * |y| < 8 off
        assert abs(d - float(gx[t, h, i])) <= 3 * 2.0 ** -11 * scale * 8


def test_nan_and_infinity_go_to_their_pairs():
    q = torch.ones(2, 1, 256, dtype=torch.bfloat16, device=DEV)
    q[0, 0, 3], q[1, 0, 200] = float("nan"), float("inf")
    got, _ = G.rope(q, None, i32([5, 6]), _freq(64))
    assert torch.isnan(got[0, 0]).nonzero().flatten().tolist() == [3, 35]
    assert torch.isinf(got[1, 0]).nonzero().flatten().tolist() == [200]


def test_nothing_to_do_and_refusals():
    f = _freq(64)
    q = _x((0, 4, 256), 14, torch.bfloat16)
    out, _ = G.rope(q, None, i32([]), f)
    assert out.shape == (0, 4, 256)
    q, k = _x((3, 4, 256), 15, torch.bfloat16), _x((3, 2, 256), 16, torch.bfloat16)
    p = i32([0, 1, 2])
    for bad in (lambda: G.rope(q.float(), k, p, f), lambda: G.rope(q, k.half(), p, f),
                lambda: G.rope(q, k, p.long(), f), lambda: G.rope(q, k, p, f.double())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: G.rope(q, k[:2], p, f), lambda: G.rope(q, k, p[:2], f), lambda: G.rope(q.cpu(), k, p, f),
                lambda: G.rope(q[..., :128], None, p, f), lambda: G.rope(q, None, p, f, k_out=k),
                lambda: G.rope(q.transpose(1, 2), None, p, f),
                lambda: G.rope(_x((3, 4, 512), 17, torch.bfloat16)[..., ::2], None, p, f)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: G.rope(q, k, p, f[:4]), lambda: G.rope(q, k, p, f[:12]),
                lambda: G.rope(q, k, p, f, q_out=torch.empty(3, 1, 256, device=DEV, dtype=q.dtype).expand(3, 4, 256)),
                lambda: G.rope(_x((3, 4 * 256 + 4), 18, torch.bfloat16)[:, 4:].view(3, 4, 256), None, p, f)):
        with pytest.raises(G.GqaError):
            bad()
    with pytest.raises(ValueError):
        G.rope_frequencies(60)
    assert G.last_device_status() == 0


def test_other_stream_and_graph():
    q, p, f = _x((64, 8, 256), 19, torch.bfloat16), i32(list(range(64))), _freq(64)
    want, _ = G.rope(q, None, p, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(q)
    with torch.cuda.stream(s):
        G.rope(q, None, p, f, q_out=out)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.rope(q, None, p, f, q_out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
