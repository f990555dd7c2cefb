"""Prompt chunks over the paged 8-bit cache against the float64 oracle on the same values."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, cu_of, i32, rows_qg
from tests.parity import assert_nonfinite_parity, assert_parity_dtype, to_f64
from tests.test_gpu_kv8_decode import LSE_TOL

pytestmark = pytest.mark.gpu


def _run(c, rows, q, g, lse=False, max_rows=None, max_kv_len=None, cu=None, **kw):
    return G.kv8_prefill(q.to(DEV), *c.device()[:4], None if g is None else g.to(DEV), i32(c.tables),
                         i32(c.lens), i32(cu or cu_of(rows)), max_rows=max_rows or max(1, max(rows)),
                         max_kv_len=max_kv_len or max(c.lens), return_lse=lse, **kw)


def _check(c, rows, Hq, seed, dtype=torch.bfloat16, gate=True, **kw):
    q, g = rows_qg(sum(rows), Hq, seed, dtype)
    out, lse = _run(c, rows, q, g if gate else None, lse=True, **kw)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g) if gate else None, c.lens, cu_of(rows))
    assert_parity_dtype(out, ref, f"kv8 prefill {rows} {c.lens}")
    assert np.abs(to_f64(lse) - rl).max(initial=0) <= LSE_TOL
    return out


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([100], [100]), ([5, 130, 1], [5, 700, 129]),
                                       ([127, 0, 129], [128, 40, 130]), ([64, 300], [1200, 300]),
                                       ([2], [2900])])
def test_parity(rows, lens, bs, dtype):
    c = Cache(lens, 2, bs, seed=141)
    _check(c, rows, 12, 142, dtype)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (24, 4), (16, 2), (16, 1), (17, 1), (10, 2), (300, 1)])
def test_head_layouts(Hq, Hkv):
    c = Cache([300, 77], Hkv, 32, seed=143)
    _check(c, [70, 77], Hq, 144)
    _check(c, [3, 1], Hq, 145, torch.float16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_many_sequences_and_a_long_one(dtype):
    """300 sequences go in two launches; one long context is cut among all pairs."""
    lens = [17 * (i % 23) + 1 for i in range(300)]
    c = Cache(lens, 1, 16, seed=146)
    _check(c, [min(n, 1 + i % 40) for i, n in enumerate(lens)], 4, 147, dtype)
    c = Cache([20000, 40], 1, 128, seed=148)
    _check(c, [33, 40], 8, 149, dtype)


U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _bounded(c, rows, Hq, seed, dtype):
    """Rows of one sequence against an error bound of every element's own.  With s the scores, w the
    probabilities and A = sum w |v| sigmoid(g), an output may be off by

        A (2 ds + u + 2 * 2^-11 + 2^-13) + F + 2^-25
                                  u: half a step of the type, for the output; 2^-11 the probabilities' own as
                                    fp16, in the sum of values (twice, beside the fp32 sum of weights); fp16's
                                    smallest half step
        ds <= (2^-16 sum |q k| + 2^-19 max |q| sum |k|) ks / 16   256 fp32 sums, and what the terms
                                    of a row's small elements of Q lose, the largest over its keys
        F = n 2^-24 max(w vs) 448   the probabilities' own step, with the values' scale, 2^-24 of the
                                    largest; a code is 448 at most
    """
    (n,) = c.lens
    q, g = rows_qg(rows, Hq, seed, dtype)
    out, lse = _run(c, [rows], q, g, lse=True)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    blocks = [c.tables[0][j // c.bs] for j in range(n)]
    qq, gg, got, gl = to_f64(q), to_f64(g), to_f64(out), to_f64(lse)
    gqa = Hq // c.Hkv
    for t in range(0, rows, max(1, rows // 9)):
        m = n - rows + t + 1
        for h in range(Hq):
            kk, vv = k[0, h // gqa, :m], v[0, h // gqa, :m]
            vs = c.vs[blocks[:m], h // gqa]
            s = kk @ qq[t, h] / 16
            w = np.exp(s - s.max())
            l = w.sum()
            w /= l
            sig = 1 / (1 + np.exp(-gg[t, h]))
            ds = ((2.0**-16 * (np.abs(kk) @ np.abs(qq[t, h]))
                   + 2.0**-19 * np.abs(qq[t, h]).max() * np.abs(kk).sum(1)) / 16).max()
            tol = (w @ np.abs(vv)) * sig * (2 * ds + U[dtype] + 2 * 2.0**-11 + 2.0**-13)
            tol += m * 2.0**-24 * (w * vs).max() * 448 + 2.0**-25
            err = np.abs(got[t, h] - (w @ vv) * sig)
            assert np.all(err <= tol), (t, h, (err / tol).max())
            assert abs(gl[t, h] - (s.max() + np.log(l))) <= ds + 1e-5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bounds_block_scales_far_apart(dtype):
    c = Cache([400], 2, 16, seed=59)
    for i, e in enumerate([-60, -7, 3, -30, -7, -20, -7, 0]):
        c.vs[c.tables[0][i]] = 2.0 ** e
        c.ks[c.tables[0][i]] = 2.0 ** [-7, -30, -7, -3, -7, -9, -40, -7][i]
    _bounded(c, 9, 8, 60, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bounds_scales_that_move_both_references(dtype):
    c = Cache([3000], 2, 64, seed=171)
    rng = np.random.RandomState(172)
    for i in range(-(-3000 // 64)):
        c.vs[c.tables[0][i]] = 2.0 ** (-6 + rng.randint(-14, 15))
        c.ks[c.tables[0][i]] = 2.0 ** (-7 + rng.randint(-2, 3))
    _bounded(c, 20, 8, 173, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bounds_ordinary_blocks(dtype):
    _bounded(Cache([2500], 2, 32, seed=174), 90, 8, 175, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_bounds_scales_that_are_no_powers_of_two_and_zeros(dtype):
    """Any finite scales of 0 and more: K's of a block 0 (its scores are 0), V's of another 0."""
    c = Cache([700], 2, 32, seed=176)
    rng = np.random.RandomState(177)
    c.ks, c.vs = (np.exp2(rng.uniform(-9, -5, c.ks.shape)).astype(np.float32).astype(np.float64) for _ in "kv")
    c.ks[c.tables[0][2]] = 0.0
    c.vs[c.tables[0][4]] = 0.0
    c.ks[c.tables[0][5]] = c.vs[c.tables[0][5]] = 0.0
    _bounded(c, 33, 8, 178, dtype)


@pytest.mark.parametrize("base", [0, 126, 127, 128, 129, 255])
def test_tile_edges(base):
    """Rows whose last keys fall on either side of a tile's end, in segments that start inside a token's heads."""
    c = Cache([base + 3, base + 87], 1, 16, seed=180)
    _check(c, [3, 87], 3, 181)
    _check(c, [2, 44], 7, 182, torch.float16)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_tail_of_many_small_probabilities_is_not_lost(dtype):
    """One key weighs e^8 times as much as each of 20,000 others (head 0), which together outweigh it."""
    n, rows = 20001, 40
    c = Cache([n], 1, 64, seed=61)
    c.k[:] = 0
    c.ks[:] = 1.0
    c.vs[:] = 2.0 ** -6
    q = torch.zeros(rows, 4, 256, dtype=dtype)
    q[:, :, 0] = torch.tensor([1.0, 0.5, 0.25, 0.0])
    c.k[c.tables[0][0], 0, 7, 0] = int(oracle.e4m3_encode(np.array([128.0]))[0])   # 8 nats over 16 * 1/16
    g = torch.zeros(rows, 4, 256, dtype=dtype)
    out, lse = _run(c, [rows], q, g, lse=True)
    k, v = c.contiguous()
    ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, rows])
    assert np.abs(to_f64(lse) - rl).max() <= LSE_TOL
    assert_parity_dtype(out, ref)


def test_no_gate_and_the_same_as_decode():
    c = Cache([70, 5, 900], 2, 16, seed=53)
    rows = [40, 5, 130]
    a = _check(c, rows, 8, 54, gate=False)
    q, _ = rows_qg(sum(rows), 8, 54)
    b = G.kv8_decode(q.to(DEV), *c.device()[:4], None, i32(c.tables), i32(c.lens), i32(cu_of(rows)))
    # each is off by 2^-8 of itself and of the values' weighted size (|v| < 4) at most, a probability's step beside
    assert (a.float() - b.float()).abs().max().item() <= 2 * 2 * 2.0 ** -8 * 4
    d = G.kv8_prefill(q.to(DEV), *c.device()[:4], None, i32(c.tables), i32(c.lens), i32(cu_of(rows)))
    assert torch.equal(a, d)


def test_rows_behind_the_last_sequence_and_skipped_ones_stay():
    c = Cache([50, 60, 70, 40], 2, 16, seed=62)
    q, g = rows_qg(9, 8, 63)
    out = torch.full((9, 8, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    lens = i32([50, 90, 70, 1])          # 1: past max_kv_len; 3: fewer keys than rows
    G.kv8_prefill(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), lens, i32([0, 2, 3, 5, 7]), max_rows=2,
                  max_kv_len=70, out=out)
    assert G.last_device_status() == 6
    k, v = c.contiguous()
    ref, _ = oracle.decode(to_f64(q[:7]), k, v, to_f64(g[:7]), [50, 60, 70, 40], [0, 2, 3, 5, 7])
    keep = [0, 1, 3, 4]
    assert_parity_dtype(out[keep], ref[keep])
    assert torch.all(out[2] == 7) and torch.all(out[5:] == 7)
    out.fill_(3)                         # no rows at all
    G.kv8_prefill(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32([50, 0, 70, 9]), i32([0] * 5), max_rows=1,
                  max_kv_len=70, out=out)
    assert G.last_device_status() == 0 and torch.all(out == 3)
    # row offsets that fall or pass T
    G.kv8_prefill(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32([50, 60, 70, 40]), i32([0, 4, 2, 11, 12]),
                  max_rows=8, max_kv_len=70, out=out)
    assert G.last_device_status() == 6 and torch.all(out[4:] == 3)
    assert not torch.any(out[:4] == 3)


def test_table_entries_outside_the_pool_read_as_zeros():
    c = Cache([40, 140], 1, 16, seed=64)
    bad = [list(t) for t in c.tables]
    bad[0][1], bad[1][2], bad[1][8] = c.N + 5, -1, 1 << 30
    for b, i in ((0, 1), (1, 2), (1, 8)):
        for pool in (c.k, c.v):
            pool[c.tables[b][i]] = 0
    q, g = rows_qg(30, 4, 65)
    k, v = c.contiguous()
    ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, 10, 30])
    c.tables = bad
    out, lse = _run(c, [10, 20], q, g, lse=True)
    assert G.last_device_status() == 6
    assert_parity_dtype(out, ref)
    assert np.abs(to_f64(lse) - rl).max() <= LSE_TOL


def test_shared_blocks_and_unused_entries():
    """Two tables name the same blocks; entries behind the last key may hold anything."""
    c = Cache([100, 100], 2, 32, seed=66)
    c.tables[1] = list(c.tables[0])
    c.tables[0][4:] = [1 << 29] * len(c.tables[0][4:])
    for pool in (c.k, c.v):
        pool[c.tables[0][3], :, 4:] = 0x7F
    q, g = rows_qg(40, 8, 67)
    q[20:], g[20:] = q[:20], g[:20]
    out = _run(c, [20, 20], q, g)
    assert G.last_device_status() == 0 and torch.equal(out[:20], out[20:])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_visible_nan_and_nonfinite_q_and_gates(dtype):
    c = Cache([200, 33], 1, 16, seed=69)
    c.v[c.tables[0][3], 0, 4, 10:20] = 0xFF                 # a NaN value in some dims
    q, g = rows_qg(34, 4, 70, dtype)
    q[1, 2, 5] = float("nan")
    q[33, 0, 9] = float("inf")
    g[0, 1, 3], g[0, 1, 4], g[30, 2, 7] = float("nan"), -float("inf"), float("inf")
    out = _run(c, [30, 4], q, g)
    k, v = c.contiguous()
    with np.errstate(all="ignore"):
        ref, _ = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, [0, 30, 34])
    assert_nonfinite_parity(out, ref)


@pytest.mark.parametrize("n,rows,Hq,Hkv", [(150, 20, 12, 2), (700, 700, 2, 2), (20000, 300, 8, 1)])
def test_a_nan_in_a_later_row(n, rows, Hq, Hkv):
    """Rows before a key with a NaN value are as if it were not there; its own row and later ones are NaN in
    its dims alone (both halves of the dims, which two CTAs hold; cut segments too)."""
    c = Cache([n], Hkv, 64, seed=71)
    q, g = rows_qg(rows, Hq, 72)
    a = _run(c, [rows], q, g)
    for i, dims in ((rows // 2, [3]), (rows - 2, [130, 255])):
        pos = n - rows + i
        for dim in dims:
            c.v[c.tables[0][pos // 64], 0, pos % 64, dim] = 0x7F
    c.k[c.tables[0][(n - 1) // 64], 0, (n - 1) % 64, 9] = 0xFF     # the last key's own
    z = _run(c, [rows], q, g)
    assert G.last_device_status() == 0
    h, i = Hq // Hkv, rows // 2
    assert torch.equal(z[:i], a[:i]) and torch.equal(z[:, h:], a[:, h:])
    assert torch.isnan(z[i:, :h, 3].float()).all()
    assert torch.isnan(z[rows - 2:, :h, [130, 255]].float()).all() and torch.isnan(z[-1, :h].float()).all()
    keep = [d for d in range(256) if d not in (3, 130, 255)]
    assert torch.equal(z[:-1, :, keep], a[:-1, :, keep])
    assert torch.equal(z[:rows - 2, :, [130, 255]], a[:rows - 2, :, [130, 255]])


def test_same_bits_again_and_alone():
    c = Cache([3000, 90, 1700], 4, 64, seed=73)
    rows = [100, 90, 33]
    q, g = rows_qg(sum(rows), 24, 74)
    a, b = _run(c, rows, q, g), _run(c, rows, q, g)
    assert torch.equal(a, b)
    q2 = q.clone()
    q2[100:190] = 5.0
    z = _run(c, rows, q2, g)
    assert torch.equal(z[:100], a[:100]) and torch.equal(z[190:], a[190:])


def test_workspace_and_output_are_kept_to():
    """Nothing is written in front of or behind the workspace and the output; a short workspace is refused."""
    c = Cache([20000, 70], 1, 64, seed=75)
    rows = [50, 70]
    q, g = rows_qg(120, 8, 76)
    want = _run(c, rows, q, g)
    n = G.kv8_prefill_workspace_size()
    ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((124, 8, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    got = _run(c, rows, q, g, workspace=ws[256:256 + n], out=out[2:122])
    assert torch.equal(got, want)
    assert torch.all(ws[:256] == 0xA5) and torch.all(ws[256 + n:] == 0xA5)
    assert torch.all(out[:2] == 9) and torch.all(out[122:] == 9)
    with pytest.raises(G.GqaError) as e:
        _run(c, rows, q, g, workspace=ws[:n - 16])
    assert e.value.code == 5
    with pytest.raises(ValueError):
        _run(c, rows, q, g, workspace=torch.empty(n, dtype=torch.uint8))
    with pytest.raises(ValueError):
        _run(c, rows, q[:, :, :128], g)
    with pytest.raises(TypeError):
        _run(c, rows, q.float(), g)


def test_two_streams_and_a_graph():
    c = Cache([9000, 300], 2, 32, seed=77)
    rows = [60, 300]
    q, g = rows_qg(360, 8, 78)
    a = _run(c, rows, q, g)
    dev, tab, lens, cu = c.device()[:4], i32(c.tables), i32(c.lens), i32(cu_of(rows))
    qd, gd = q.to(DEV), g.to(DEV)
    call = lambda ws, out: G.kv8_prefill(qd, *dev, gd, tab, lens, cu, max_rows=300, max_kv_len=9000,  # noqa: E731
                                         workspace=ws, out=out)
    ws = [torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8, device=DEV) for _ in range(2)]
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
    assert torch.equal(outs[0], _run(c, rows, q.flip(0), g)) and G.last_device_status() == 0


def test_a_prompt_in_chunks_is_the_whole_prompt():
    """Fork, plan, rope, append, attention of the chunk, one step of decode, free, compact: a server's round over a
    shared prefix, the cache and every row's output against the oracle."""
    B, Hq, Hkv, bs, N, width, rot = 4, 8, 2, 32, 60, 16, 64
    gen = torch.Generator().manual_seed(80)
    o = dict(tables=[[-1] * width for _ in range(B)], n=[0] * B, free=list(range(N)), lens=[0] * B, shares=[0] * N)
    pools = [np.zeros((N, Hkv, bs, 256), dtype=np.uint8) for _ in "kv"]
    scales = [np.ones((N, Hkv)) for _ in "kv"]
    d = {k: i32(v) for k, v in o.items()}
    d["fc"] = i32([N])
    dp = [torch.from_numpy(p).to(DEV).view(torch.float8_e4m3fn) for p in pools]
    ds = [torch.ones(N, Hkv, device=DEV) for _ in "kv"]
    freq, _ = G.rope_frequencies(rot)
    ws = torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8, device=DEV)

    def step(rows):
        T, cu = sum(rows), cu_of(rows)
        x = torch.randn(T, Hq + 2 * Hkv, 256, generator=gen).to(DEV, torch.bfloat16)
        g = torch.randn(T, Hq, 256, generator=gen).to(DEV, torch.bfloat16)
        pos = [o["lens"][b] + i for b in range(B) for i in range(rows[b])]
        q, k = G.rope(x[:, :Hq], x[:, Hq:Hq + Hkv], i32(pos), freq)
        v = x[:, Hq + Hkv:].contiguous()
        slots, d["lens"] = G.block_plan(d["lens"], i32(cu), d["tables"], d["n"], d["free"], d["fc"], bs, T)
        G.kv8_append(k, v, slots, *dp, *ds)
        attend = G.kv8_prefill if max(rows) > 1 else G.kv8_decode
        kw = dict(workspace=ws) if max(rows) > 1 else {}
        out = attend(q, *dp, *ds, g, d["tables"], d["lens"], i32(cu), max_rows=max(rows), max_kv_len=width * bs, **kw)
        os_, o["lens"], _ = oracle.block_plan(o["lens"], rows, o["tables"], o["n"], o["free"], bs, T)
        for p, s, y in zip(pools, scales, (k, v)):
            at = 0
            for r in rows:
                oracle.kv8_append(p, s, to_f64(y[at:at + r]), os_[at:at + r], bs)
                at += r
        kk, vv = (oracle.kv8_contiguous(p, s, o["tables"], o["lens"], bs) for p, s in zip(pools, scales))
        live = [b for b in range(B) if rows[b]]
        ref, _ = oracle.decode(to_f64(q), kk[live], vv[live], to_f64(g), [o["lens"][b] for b in live],
                               cu_of([rows[b] for b in live]))
        assert_parity_dtype(out, ref, f"step {rows}")
        check()

    def check():
        assert G.last_device_status() == 0
        assert d["tables"].tolist() == o["tables"] and d["shares"].tolist() == o["shares"]
        assert d["lens"].tolist() == o["lens"] and d["fc"].item() == len(o["free"])
        for t, s, p, sc in zip(dp, ds, pools, scales):
            got = oracle.kv8_contiguous(t.view(torch.uint8).cpu().numpy(), s.double().cpu().numpy(), o["tables"],
                                        o["lens"], bs)
            assert np.array_equal(got, oracle.kv8_contiguous(p, sc, o["tables"], o["lens"], bs))

    step([150, 0, 0, 0])
    copies, _ = oracle.block_fork([0, 0, 0], [1, 2, 3], [150, 100, 64], o["lens"], o["tables"], o["n"], o["free"],
                                  o["shares"], bs)
    oracle.kv8_copy(copies, pools, scales)
    got = G.block_fork(i32([0, 0, 0]), i32([1, 2, 3]), i32([150, 100, 64]), d["lens"], d["tables"], d["n"], d["free"],
                       d["fc"], d["shares"], bs)
    assert got.tolist() == copies
    G.kv8_copy(got, *dp, *ds)
    check()
    step([0, 37, 70, 5])
    step([1, 1, 1, 1])
    o["lens"][0], o["lens"][2] = 0, 40              # the parent ends, a child is cut below its fork
    d["lens"] = i32(o["lens"])
    oracle.block_free(o["lens"], o["tables"], o["n"], o["free"], o["shares"], bs)
    G.block_free(d["lens"], d["tables"], d["n"], d["free"], d["fc"], d["shares"], bs)
    check()
    o["tables"], o["free"], o["shares"], _, copies = oracle.block_compact(o["tables"], o["n"], o["free"], o["shares"], N,
                                                                         bs)
    oracle.kv8_copy(copies, pools, scales)
    d["tables"], d["free"], d["shares"], _, got = G.block_compact(d["tables"], d["n"], d["free"], d["fc"], d["shares"],
                                                                  bs)
    G.kv8_copy(got, *dp, *ds)
    check()
    step([20, 1, 33, 0])
    step([1, 1, 1, 1])


@pytest.mark.parametrize("Hkv,rows,lens,max_kv_len", [
    (2, [20] * 6, [1280] * 6, None),                       # ten tiles
    (2, [20] * 6, [1281] * 6, None),                       # one more
    (2, [20] * 6, [1409, 1537, 1665, 20, 100, 1300], None),
    (2, [45, 0, 30, 1, 200], [1290, 70, 500, 1, 1500], None),
    (1, [30] * 30, [700] * 30, 5000),                      # a bound far above the lengths
    (1, [64] + [1] * 9, [1700] + [40] * 9, None),
    (4, [9] * 19, [900 + 7 * i for i in range(19)], None),   # 76 segments
    (7, [9] * 11, [800 + 7 * i for i in range(11)], None),   # 77
    (1, [40, 40], [9000, 2600], None),
])
def test_short_segments_whole_and_cut(Hkv, rows, lens, max_kv_len):
    """Segments on either side of where they are shared between pairs, after a call that cut all."""
    ws = torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8, device=DEV)
    _check(Cache([20000], 1, 128, seed=181), [30], 8, 182, workspace=ws)
    c = Cache(lens, Hkv, 64, seed=183, room=max(0, (max_kv_len or 0) - min(lens)))
    _check(c, rows, 6 * Hkv, 184, max_kv_len=max_kv_len, workspace=ws)


def test_captured_steps_on_a_growing_cache_and_a_shared_workspace():
    """A captured step (plan, rope, append, attention of its rows) grows the cache at each replay as eager calls do; a
    second graph with the same workspace, whose segments are cut where the first's are whole, runs in between."""
    B, Hq, Hkv, bs, N, width = 2, 8, 2, 64, 40, 20
    gen = torch.Generator().manual_seed(190)
    rows = [70, 45]
    T, cu = sum(rows), i32(cu_of(rows))
    x = torch.randn(T, Hq + 2 * Hkv, 256, generator=gen).to(DEV, torch.bfloat16)
    g = torch.randn(T, Hq, 256, generator=gen).to(DEV, torch.bfloat16)
    v = x[:, Hq + Hkv:].contiguous()
    freq, scale = G.rope_frequencies(64)
    ws = torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8, device=DEV)

    def fresh():
        return dict(lens=i32([0] * B), tables=i32([[-1] * width] * B), n=i32([0] * B), free=i32(list(range(N))),
                    fc=i32([N]), pos=torch.cat([torch.arange(r) for r in rows]).to(DEV, torch.int32),
                    pools=[torch.zeros(N, Hkv, bs, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
                           for _ in "kv"], scales=[torch.ones(N, Hkv, device=DEV) for _ in "kv"],
                    slots=i32([0] * T), new=i32([0] * B), out=torch.zeros(T, Hq, 256, dtype=torch.bfloat16, device=DEV))

    by_seq = i32([b for b in range(B) for _ in range(rows[b])])
    grow = i32(rows)[by_seq.long()]

    def step(s):
        G.block_plan(s["lens"], cu, s["tables"], s["n"], s["free"], s["fc"], bs, T, slots=s["slots"],
                     kv_lens_out=s["new"])
        q, k = G.rope(x[:, :Hq], x[:, Hq:Hq + Hkv], s["pos"], freq, scale=scale)
        G.kv8_append(k, v, s["slots"], *s["pools"], *s["scales"])
        G.kv8_prefill(q, *s["pools"], *s["scales"], g, s["tables"], s["new"], cu, max_rows=max(rows),
                      max_kv_len=width * bs, workspace=ws, out=s["out"])
        s["lens"].copy_(s["new"])
        s["pos"].add_(grow)

    c = Cache([9000, 300], 2, 32, seed=191)
    q2, g2 = (t.to(DEV) for t in rows_qg(360, 8, 192))
    dev, tab, lens2, cu2 = c.device()[:4], i32(c.tables), i32(c.lens), i32(cu_of([60, 300]))
    other = lambda out: G.kv8_prefill(q2, *dev, g2, tab, lens2, cu2, max_rows=300, max_kv_len=9000,  # noqa: E731
                                      workspace=ws, out=out)
    want2 = other(torch.zeros_like(q2)).clone()
    a, b, out2 = fresh(), fresh(), torch.zeros_like(q2)
    step(fresh())                                          # (everything is loaded before the captures)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        step(a)
    with torch.cuda.graph(second):
        other(out2)
    for _ in range(5):
        out2.zero_()
        first.replay()
        second.replay()
        step(b)
        torch.cuda.synchronize()
        assert torch.equal(a["out"], b["out"]) and torch.equal(out2, want2)
        assert a["lens"].tolist() == b["lens"].tolist() and torch.equal(a["tables"], b["tables"])
    assert G.last_device_status() == 0 and a["lens"].tolist() == [350, 225]
