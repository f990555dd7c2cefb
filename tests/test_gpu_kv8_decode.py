"""Attention over the paged 8-bit cache against the float64 oracle on the same values."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from synth import inputs as S
from tests.kv8_cases import DEV, Cache, cu_of, f8, i32, rows_qg
from tests.parity import assert_nonfinite_parity, assert_parity_dtype, to_f64

pytestmark = pytest.mark.gpu

# lse = m + ln l in fp32 from scores of 256 products: |s| error <= 256 * 2^-24 * sum|q k| / 16,
# sum |q k| <= |q| |k| ~ 16 * 16 (unit normal values; the caches' are up to 4 times larger, so 2^-8 of
# room), plus exp / log of a few 2^-22: 256 * 2^-24 * 64 * 16 / 16 = 1e-3.
LSE_TOL = 1e-3


def _run(c, rows, q, g, mask=None, lse=False, max_rows=None, max_kv_len=None, T=None, **kw):
    return G.kv8_decode(q.to(DEV), *c.device()[:4], None if g is None else g.to(DEV),
                        i32(c.tables), i32(c.lens), i32(cu_of(rows)),
                        tree_mask=None if mask is None else torch.tensor(mask, dtype=torch.int64, device=DEV),
                        max_rows=max_rows or max(1, max(rows)), max_kv_len=max_kv_len or max(c.lens),
                        return_lse=lse, **kw)


def _check(c, rows, Hq, seed, dtype=torch.bfloat16, mask=None, gate=True, **kw):
    q, g = rows_qg(sum(rows), Hq, seed, dtype)
    if not gate:
        g = None
    out, lse = _run(c, rows, q, g, mask, lse=True, **kw)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    gg = None if g is None else to_f64(g)
    if mask is None:
        ref, rl = oracle.decode(to_f64(q), k, v, gg, c.lens, cu_of(rows))
    else:
        ref, rl = oracle.decode_tree(to_f64(q), k, v, gg, c.lens, cu_of(rows), mask)
    assert_parity_dtype(out, ref, f"kv8 {rows} {c.lens}")
    got = to_f64(lse)
    assert np.array_equal(np.isinf(got), np.isinf(rl))
    fin = np.isfinite(rl)
    assert np.abs(got[fin] - rl[fin]).max(initial=0) <= LSE_TOL
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 15, 16, 17], [127, 128, 129, 1], [1000, 63, 2049]])
def test_decode_parity(lens, bs, dtype):
    c = Cache(lens, 2, bs, seed=41)
    _check(c, [1] * len(lens), 12, 42, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (24, 4), (16, 2), (16, 1), (17, 1), (40, 1),
                                    (128, 1), (10, 2)])
def test_decode_head_layouts(Hq, Hkv):
    c = Cache([300, 77], Hkv, 32, seed=43)
    _check(c, [1, 1], Hq, 44)
    _check(c, [3, 1], Hq, 45, torch.float16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,lens", [([2, 3, 1], [2, 300, 129]), ([4, 0, 4], [4, 5, 600]),
                                       ([33, 7], [900, 7]), ([130], [400]),
                                       ([40, 3, 64], [700, 260, 64])])
def test_chain_verify(rows, lens, dtype):
    c = Cache(lens, 2, 64, seed=46)
    _check(c, rows, 12, 47, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,lens", [([6, 4], [300, 1500]), ([32, 1, 9], [900, 1, 9]), ([64], [64]),
                                       ([64, 64], [200, 129])])
def test_tree_verify(rows, lens, dtype):
    c = Cache(lens, 2, 32, seed=48)
    mask = S.random_tree_masks(rows, 49)
    _check(c, rows, 16, 50, dtype, mask=[m - (1 << 64) if m >> 63 else m for m in mask])


def test_tree_rows_that_see_nothing():
    """A mask of no bits and no earlier key: zeros and lse -inf; others of the batch as usual."""
    c = Cache([3, 40], 1, 16, seed=51)
    mask = [0, 2, 0, 1, 0]
    q, g = rows_qg(5, 4, 52)
    out, lse = _run(c, [3, 2], q, g, mask, lse=True)
    k, v = c.contiguous()
    ref, rl = oracle.decode_tree(to_f64(q), k, v, to_f64(g), c.lens, [0, 3, 5], mask)
    assert_parity_dtype(out, ref)
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -float("inf"))
    assert torch.all(out[2] == 0) and not torch.any(torch.isinf(lse[3:]))


def test_no_gate_and_no_cu_rows():
    c = Cache([70, 5, 900], 2, 16, seed=53)
    a = _check(c, [1, 1, 1], 8, 54, gate=False)
    q, _ = rows_qg(3, 8, 54)
    b = G.kv8_decode(q.to(DEV), *c.device()[:4], None, i32(c.tables), i32(c.lens))
    assert torch.equal(a, b)


def test_long_sequences_and_many():
    c = Cache([20000, 33000], 1, 128, seed=55)
    _check(c, [1, 1], 8, 56)
    c = Cache([17 * (i % 23) + 1 for i in range(300)], 1, 16, seed=57)
    _check(c, [1] * 300, 4, 58)


@pytest.mark.parametrize("rows", [1, 9])        # 4 packed rows, and 36: the kernel for many
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block_scales_far_apart(dtype, rows):
    """Blocks whose values differ by many powers of two: a sink block of tiny values that takes nearly
    all probability next to large ones, and keys whose scores differ by tens."""
    c = Cache([400], 2, 16, seed=59)
    for i, e in enumerate([-60, -7, 3, -30, -7, -20, -7, 0]):
        c.vs[c.tables[0][i]] = 2.0 ** e
        c.ks[c.tables[0][i]] = 2.0 ** [-7, -30, -7, -3, -7, -9, -40, -7][i]
    q, g = rows_qg(rows, 8, 60, dtype)
    out, lse = _run(c, [rows], q, g, lse=True)
    k, v = c.contiguous()
    ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, rows])
    # scores reach 2^4 times a usual one: their fp32 error is 16 * LSE_TOL at most
    tol = 16 * LSE_TOL
    assert np.abs(to_f64(lse) - rl).max() <= tol
    u = torch.finfo(dtype).eps / 2
    scale = np.abs(ref).max()
    assert np.abs(to_f64(out) - ref).max() <= scale * (4 * u + 2 * tol)


@pytest.mark.parametrize("rows", [1, 16])       # 4 packed rows, and 64: the kernel for many
def test_a_tail_of_many_small_probabilities_is_not_lost(rows):
    """One key weighs e^8 times as much as each of 20,000 others (head 0), which together outweigh it."""
    n = 20001
    c = Cache([n], 1, 64, seed=61)
    c.k[:] = 0
    c.ks[:] = 1.0
    c.vs[:] = 2.0 ** -6
    q = torch.zeros(rows, 4, 256, dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 0.5, 0.25, 0.0])
    c.k[c.tables[0][0], 0, 7, 0] = int(oracle.e4m3_encode(np.array([128.0]))[0])   # 8 nats over 16 * 1/16
    g = torch.zeros(rows, 4, 256, dtype=torch.bfloat16)
    for dtype in (torch.bfloat16, torch.float16):
        out, lse = _run(c, [rows], q.to(dtype), g.to(dtype), lse=True)
        k, v = c.contiguous()
        ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, rows])
        assert np.abs(to_f64(lse) - rl).max() <= LSE_TOL
        assert_parity_dtype(out, ref)


def test_rows_behind_the_last_sequence_and_skipped_ones_stay():
    c = Cache([50, 60, 70], 2, 16, seed=62)
    q, g = rows_qg(8, 8, 63)
    out = torch.full((8, 8, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    lens = i32([50, 90, 70])             # past max_kv_len: sequence 1 is skipped
    G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), lens, i32([0, 2, 3, 5]),
                 max_rows=2, max_kv_len=70, out=out)
    assert G.last_device_status() == 6
    k, v = c.contiguous()
    ref, _ = oracle.decode(to_f64(q[:5]), k, v, to_f64(g[:5]), [50, 60, 70], [0, 2, 3, 5])
    keep = [0, 1, 3, 4]
    assert_parity_dtype(out[keep], ref[keep])
    assert torch.all(out[2] == 7) and torch.all(out[5:] == 7)
    # all sequences empty
    out.fill_(3)
    G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32([50, 0, 70]),
                 i32([0, 0, 0, 0]), max_rows=1, max_kv_len=70, out=out)
    assert G.last_device_status() == 0 and torch.all(out == 3)


def test_table_entries_outside_the_pool_are_recorded():
    c = Cache([40, 40], 1, 16, seed=64)
    c.tables[0][1] = c.N + 5
    c.tables[1][2] = -1
    q, g = rows_qg(2, 4, 65)
    out = _run(c, [1, 1], q, g)
    assert G.last_device_status() == 6 and torch.isfinite(out.float()).all()


def test_hidden_nan_never_shows():
    """NaN codes and scales in places that a row does not see - stale rows of its last block (every
    test's caches hold them), other blocks, and draft rows hidden from it - change no bit."""
    rows, lens = [5, 9], [45, 140]
    mask = S.random_tree_masks(rows, 66)
    cu = cu_of(rows)
    for hkv, hq, bs in ((2, 8, 32), (1, 20, 16)):
        c = Cache(lens, hkv, bs, seed=67)
        q, g = rows_qg(sum(rows), hq, 68)
        a = _run(c, rows, q, g, mask)
        hidden = []      # (sequence, draft row) hidden from at least one other row
        for b, r in enumerate(rows):
            for k in range(r):
                if any(not (mask[cu[b] + i] >> k) & 1 for i in range(r)):
                    hidden.append((b, k))
        b, k = hidden[len(hidden) // 2]
        pos = lens[b] - rows[b] + k
        for pool in (c.k, c.v):
            pool[c.tables[b][pos // bs], :, pos % bs] = 0x7F
        z = _run(c, rows, q, g, mask)
        assert G.last_device_status() == 0
        for bb in range(2):
            for i in range(rows[bb]):
                t = cu[bb] + i
                if bb == b and (mask[t] >> k) & 1:
                    assert torch.isnan(z[t].float()).all()
                else:
                    assert torch.equal(z[t], a[t]), (b, k, t)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_visible_nan_and_nonfinite_q_and_gates(dtype):
    c = Cache([200, 33], 1, 16, seed=69)
    c.v[c.tables[0][3], 0, 4, 10:20] = 0xFF                 # a NaN value in some dims
    q, g = rows_qg(4, 4, 70, dtype)
    q[1, 2, 5] = float("nan")
    q[3, 0, 9] = float("inf")
    g[0, 1, 3], g[0, 1, 4], g[2, 2, 7] = float("nan"), -float("inf"), float("inf")
    out = _run(c, [2, 2], q, g)
    k, v = c.contiguous()
    with np.errstate(all="ignore"):
        ref, _ = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, 2, 4])
    assert_nonfinite_parity(out, ref)


def test_chain_rows_and_a_nan_in_a_later_draft():
    """Chain rows before a draft with a NaN value are as if it were not there; the draft's own row and
    later ones are NaN in its dims alone."""
    c = Cache([150], 2, 64, seed=71)
    q, g = rows_qg(20, 12, 72)
    a = _run(c, [20], q, g)
    pos = 150 - 20 + 11
    c.v[c.tables[0][pos // 64], 0, pos % 64, 3] = 0x7F
    z = _run(c, [20], q, g)
    assert torch.equal(z[:11], a[:11]) and torch.equal(z[:, 6:], a[:, 6:])
    assert torch.isnan(z[11:, :6, 3].float()).all()
    keep = [d for d in range(256) if d != 3]
    assert torch.isfinite(z[:, :, keep].float()).all()


def test_same_bits_again_and_alone():
    """Two runs agree bit for bit; a sequence's rows do not depend on the batch's other values."""
    c = Cache([3000, 90, 1700], 4, 64, seed=73)
    q, g = rows_qg(3, 24, 74)
    a, b = _run(c, [1, 1, 1], q, g), _run(c, [1, 1, 1], q, g)
    assert torch.equal(a, b)
    q2 = q.clone()
    q2[1] = 5.0
    z = _run(c, [1, 1, 1], q2, g)
    assert torch.equal(z[0], a[0]) and torch.equal(z[2], a[2])


def test_workspace_too_small_and_tree_limits():
    c = Cache([100], 1, 16, seed=75)
    q, g = rows_qg(1, 4, 76)
    with pytest.raises(G.GqaError) as e:
        _run(c, [1], q, g, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == 5
    with pytest.raises(G.GqaError) as e:
        _run(c, [1], q, g, mask=[1], max_rows=65)
    assert e.value.code == 2


def test_other_stream_graph_and_two_workspaces():
    c = Cache([900, 300], 2, 32, seed=77)
    q, g = rows_qg(2, 8, 78)
    a = _run(c, [1, 1], q, g)
    dev, tab, lens, cu = c.device()[:4], i32(c.tables), i32(c.lens), i32([0, 1, 2])
    qd, gd = q.to(DEV), g.to(DEV)
    call = lambda ws, out: G.kv8_decode(qd, *dev, gd, tab, lens, cu, max_rows=1, max_kv_len=900,  # noqa: E731
                                        workspace=ws, out=out)
    size = G.kv8_workspace_size(2, 2, 8, 2, 1, 900)
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in range(2)]
    outs = [torch.zeros_like(qd) for _ in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):                                     # two at once
        for s, w, o in zip(streams, ws, outs):
            with torch.cuda.stream(s):
                call(w, o)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a) and torch.equal(outs[1], a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws[0], outs[0])
    outs[0].zero_()
    qd.copy_(q.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    b = _run(c, [1, 1], q.flip(0), g)
    assert torch.equal(outs[0], b) and G.last_device_status() == 0


def test_a_whole_step_in_one_graph():
    """Plan, append and decode captured behind copies and in front of them, then replayed with other
    lengths and rows: each replay equals the same calls made eagerly on a copy of the state."""
    B, Hq, Hkv, bs, N, width = 4, 12, 2, 32, 40, 8
    gen = torch.Generator().manual_seed(90)
    pool = lambda: torch.zeros(N, Hkv, bs, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)  # noqa: E731

    def state():
        return dict(tables=i32([[-1] * width] * B), n=i32([0] * B), free=i32(list(range(N))), fc=i32([N]),
                    lens=i32([0] * B), k=pool(), v=pool(), ks=torch.ones(N, Hkv, device=DEV),
                    vs=torch.ones(N, Hkv, device=DEV))

    T = 8
    cu, out = i32([0] * (B + 1)), torch.zeros(T, Hq, 256, dtype=torch.bfloat16, device=DEV)
    kn, vn = (torch.zeros(T, Hkv, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    q, g = (torch.zeros(T, Hq, 256, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    src = [torch.zeros_like(x) for x in (kn, vn, q, g, cu)]
    ws = torch.empty(G.kv8_workspace_size(B, T, Hq, Hkv, T, width * bs), dtype=torch.uint8, device=DEV)
    last = torch.zeros_like(out)

    def step(s, dst):
        for a, b in zip((kn, vn, q, g, cu), src):
            a.copy_(b)
        slots, lens = G.block_plan(s["lens"], cu, s["tables"], s["n"], s["free"], s["fc"], bs, T)
        G.kv8_append(kn, vn, slots, s["k"], s["v"], s["ks"], s["vs"])
        G.kv8_decode(q, s["k"], s["v"], s["ks"], s["vs"], g, s["tables"], lens, cu, max_rows=T,
                     max_kv_len=width * bs, workspace=ws, out=dst)
        s["lens"].copy_(lens)
        last.copy_(dst)

    a, b = state(), state()
    eager = torch.zeros_like(out)
    step(state(), eager)                      # first use of every kernel, outside the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a, out)
    for key in a:                             # (capture runs nothing)
        a[key].view(torch.uint8).copy_(b[key].view(torch.uint8))
    for rows in ([3, 1, 4, 0], [1, 1, 1, 1], [0, 2, 0, 6], [1, 0, 5, 1], [2, 2, 2, 2]):
        fill = [torch.randn(x.shape, generator=gen).to(x.dtype) for x in (kn, vn, q, g)]
        for d, x in zip(src, fill + [torch.tensor(cu_of(rows), dtype=torch.int32)]):
            d.copy_(x)
        out.zero_(), eager.zero_()
        graph.replay()
        got = last.clone()
        step(b, eager)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
        for key in a:
            assert torch.equal(a[key].view(torch.uint8), b[key].view(torch.uint8)), key
    assert G.last_device_status() == 0


def test_rounds_of_serving():
    """Plan, append, decode, a tree of drafts, keep, and the next step, all captured state on the GPU:
    the cache equals the oracle's after every step, the rows its attention's."""
    B, Hq, Hkv, bs, N, width = 3, 8, 2, 16, 40, 12
    rng = np.random.RandomState(80)
    gen = torch.Generator().manual_seed(80)
    o = dict(tables=[[-1] * width for _ in range(B)], n=[0] * B, free=list(range(N)), lens=[0] * B)
    pools = [np.zeros((N, Hkv, bs, 256), dtype=np.uint8) for _ in range(2)]
    scales = [np.ones((N, Hkv)) for _ in range(2)]
    d = dict(tables=i32(o["tables"]), n=i32(o["n"]), free=i32(o["free"]), fc=i32([N]), lens=i32(o["lens"]))
    dp = [f8(p) for p in pools]
    ds = [torch.ones(N, Hkv, device=DEV) for _ in range(2)]
    plans = [([37, 1, 16], None), ([1, 1, 1], None), ([5, 9, 1], True), ([1, 1, 1], None),
             ([1, 20, 2], True), ([1, 1, 1], None)]
    for rows, tree in plans:
        T, cu = sum(rows), cu_of(rows)
        kn, vn = (torch.randn(T, Hkv, 256, generator=gen).to(torch.bfloat16) for _ in range(2))
        q, g = rows_qg(T, Hq, int(rng.randint(1 << 30)))
        slots, lens = G.block_plan(d["lens"], i32(cu), d["tables"], d["n"], d["free"], d["fc"], bs, T)
        G.kv8_append(kn.to(DEV), vn.to(DEV), slots, *dp, *ds)
        mask = S.random_tree_masks(rows, int(rng.randint(1000))) if tree else None
        out = G.kv8_decode(q.to(DEV), *dp, *ds, g.to(DEV), d["tables"], lens, i32(cu),
                           tree_mask=None if mask is None else torch.tensor(mask, device=DEV),
                           max_rows=max(rows), max_kv_len=width * bs)
        oslots, olens, _ = oracle.block_plan(o["lens"], rows, o["tables"], o["n"], o["free"], bs, T)
        for p, s, x in zip(pools, scales, (kn, vn)):
            at = 0
            for r in rows:       # the oracle takes a sequence at a time
                oracle.kv8_append(p, s, x[at:at + r].double().numpy(), oslots[at:at + r], bs)
                at += r
        k, v = (oracle.kv8_contiguous(p, s, o["tables"], olens, bs) for p, s in zip(pools, scales))
        if mask is None:
            ref, _ = oracle.decode(to_f64(q), k, v, to_f64(g), olens, cu)
        else:
            ref, _ = oracle.decode_tree(to_f64(q), k, v, to_f64(g), olens, cu, mask)
        assert_parity_dtype(out, ref, f"step {rows}")
        if tree:
            keep = [sorted(rng.choice(r, size=rng.randint(0, r + 1), replace=False).tolist()) for r in rows]
            new = torch.empty_like(lens)
            G.kv8_keep(*dp, *ds, d["tables"], lens, i32(cu), i32(sum(keep, [])),
                       i32(cu_of([len(x) for x in keep])), new)
            for p, s in zip(pools, scales):
                oracle.kv8_keep(p, s, o["tables"], olens, rows, keep, bs)
            olens, lens = [n - r + len(x) for n, r, x in zip(olens, rows, keep)], new
            assert lens.tolist() == olens
        o["lens"], d["lens"] = olens, lens
        assert G.last_device_status() == 0
        k, v = (oracle.kv8_contiguous(p, s, o["tables"], olens, bs) for p, s in zip(pools, scales))
        for t, s, ref in zip(dp, ds, (k, v)):
            got = oracle.kv8_contiguous(t.view(torch.uint8).cpu().numpy(), s.double().cpu().numpy(),
                                        d["tables"].tolist(), olens, bs)
            assert np.array_equal(got, ref)
