"""The paged 8-bit cache where calls meet: many short sequences on one CTA, pools past 2^32 bytes,
guard bands, other streams, memory, and the ends of the ranges."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from synth import inputs as S
from tests.kv8_cases import DEV, Cache, codes_of, cu_of, f8, i32, rows_qg
from tests.parity import assert_nonfinite_parity, assert_parity_dtype, to_f64

pytestmark = pytest.mark.gpu


def _call(c, rows, q, g, dev=None, mask=None, **kw):
    dev = dev or c.device()[:4]
    return G.kv8_decode(q, *dev, g, i32(c.tables), i32(c.lens), i32(cu_of(rows)), tree_mask=mask,
                        max_rows=max(rows), max_kv_len=max(c.lens), **kw)


def _ref(c, rows, q, g, mask=None):
    k, v = c.contiguous()
    if mask is None:
        return oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, cu_of(rows))[0]
    return oracle.decode_tree(to_f64(q), k, v, to_f64(g), c.lens, cu_of(rows), mask)[0]


# 8, 20, 28 and 40 packed rows: one kernel each
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("Hq,rows", [(16, 2), (16, 5), (16, 7), (32, 5)])
def test_many_sequences_of_one_tile(Hq, rows, dtype):
    """A CTA goes through several segments of a single tile, one after another: each row's result is
    its own, every time."""
    lens = [rows + (37 * i) % (128 - rows) for i in range(250)]
    c = Cache(lens, 4, 16, seed=101)
    rr = [rows] * len(lens)
    q, g = rows_qg(sum(rr), Hq, 102, dtype)
    dev, qd, gd = c.device()[:4], q.to(DEV), g.to(DEV)
    first = _call(c, rr, qd, gd, dev)
    assert_parity_dtype(first, _ref(c, rr, q, g))
    ws = torch.empty(G.kv8_workspace_size(len(lens), sum(rr), Hq, 4, rows, max(lens)),
                     dtype=torch.uint8, device=DEV)
    for _ in range(30):
        assert torch.equal(_call(c, rr, qd, gd, dev, workspace=ws), first)
    assert G.last_device_status() == 0


def test_more_sequences_than_one_launch_takes():
    """600 sequences are scheduled in three launches: chains and trees, some of them idle."""
    rows = [(i * 7) % 4 for i in range(600)]
    lens = [r + (i * 131) % 700 for i, r in enumerate(rows)]
    c = Cache(lens, 1, 64, seed=103)
    q, g = rows_qg(sum(rows), 8, 104)
    out = _call(c, rows, q.to(DEV), g.to(DEV))
    assert_parity_dtype(out, _ref(c, rows, q, g))
    mask = S.random_tree_masks(rows, 105)
    out = _call(c, rows, q.to(DEV), g.to(DEV), mask=torch.tensor(mask, dtype=torch.int64, device=DEV))
    assert_parity_dtype(out, _ref(c, rows, q, g, mask))
    assert G.last_device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 3, 4, 5, 9])
@pytest.mark.parametrize("n", [127, 128, 129, 255, 256, 257])
def test_ends_of_tiles(n, rows, dtype):
    c = Cache([n, n + 128 * 9, rows], 2, 128, seed=106)
    q, g = rows_qg(3 * rows, 16, 107, dtype)
    out = _call(c, [rows] * 3, q.to(DEV), g.to(DEV))
    assert_parity_dtype(out, _ref(c, [rows] * 3, q, g))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_nonfinite_rows_in_the_kernel_for_many(dtype):
    c = Cache([200, 40], 1, 16, seed=108)
    c.v[c.tables[0][3], 0, 4, 10:20] = 0xFF
    c.k[c.tables[1][1], 0, 2, 7] = 0x7F               # a key that every row of sequence 1 sees
    q, g = rows_qg(22, 4, 109, dtype)
    q[1, 2, 5], q[9, 0, 9] = float("nan"), float("inf")
    g[0, 1, 3], g[2, 2, 7] = float("nan"), float("inf")
    rows = [12, 10]
    out = _call(c, rows, q.to(DEV), g.to(DEV))
    with np.errstate(all="ignore"):
        ref = _ref(c, rows, q, g)
    assert_nonfinite_parity(out, ref)


def test_pools_past_2_to_the_32_bytes():
    """Blocks behind the 2^32-byte mark of a pool give the bits that the same blocks of a small one do."""
    Hkv, bs, N = 2, 64, 160000                          # 5.2e9 bytes each of K and V
    lens, rows = [300, 77], [5, 3]
    c = Cache(lens, Hkv, bs, seed=110, room=40)
    small = c.device()
    # block i of the small pool lies at N - c.N + i; the last block of the pool is among them
    at = N - c.N
    big = [torch.zeros(N, Hkv, bs, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
           for _ in "kv"] + [torch.ones(N, Hkv, device=DEV) for _ in "kv"]
    for b, s in zip(big, small):
        b[at:].view(torch.uint8 if b.dtype != torch.float32 else b.dtype).copy_(
            s.view(torch.uint8 if s.dtype != torch.float32 else s.dtype))
    big_tab = torch.where(small[4] >= 0, small[4] + at, small[4])
    assert at * Hkv * bs * 256 > 1 << 32

    def step(pools, tables, base):
        k, v = (torch.randn(sum(rows), Hkv, 256, generator=torch.Generator().manual_seed(s)).bfloat16().to(DEV)
                for s in (111, 112))
        slots = []
        for b, r in enumerate(rows):
            slots += [(base + c.tables[b][j // bs]) * bs + j % bs for j in range(lens[b], lens[b] + r)]
        G.kv8_append(k, v, i32(slots), *pools)
        new = i32([n + r for n, r in zip(lens, rows)])
        outs = []
        for Hq in (4, 16):                              # 10 and 40 packed rows
            q, g = (x.to(DEV) for x in rows_qg(sum(rows), Hq, 113))
            outs.append(G.kv8_decode(q, *pools, g, tables, new, i32(cu_of(rows)), max_rows=5, max_kv_len=310))
        G.kv8_keep(*pools, tables, new, i32(cu_of(rows)), i32([1, 4, 0, 2]), i32([0, 2, 4]))
        return outs

    a, b = step(small[:4], small[4], 0), step(big, big_tab, at)
    assert G.last_device_status() == 0
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    for x, y in zip(small[:4], big):
        assert torch.equal(x.view(torch.uint8), y[at:].contiguous().view(torch.uint8))
    assert not big[0][:at].view(torch.int64).any() and torch.all(big[2][:at] == 1)


@pytest.mark.parametrize("Hq,rows", [(4, 2), (8, 4), (16, 6)])
def test_nothing_is_written_around_the_outputs(Hq, rows):
    """Bands around out, lse and the workspace keep their bytes, and the cache all of its own."""
    c = Cache([500, 64, 7 + rows], 1, 32, seed=114)
    q, g = (x.to(DEV) for x in rows_qg(3 * rows, Hq, 115))
    dev = c.device()
    before = [t.clone() for t in dev]
    size = G.kv8_workspace_size(3, 3 * rows, Hq, 1, rows, 500)
    ws = torch.full((size + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    out = torch.full((3 * rows + 2, Hq, 256), 7.0, dtype=q.dtype, device=DEV)
    _call(c, [rows] * 3, q, g, dev[:4], workspace=ws[256:256 + size], out=out[1:-1])
    assert torch.all(out[0] == 7) and torch.all(out[-1] == 7)
    assert torch.all(ws[:256] == 0xA5) and torch.all(ws[256 + size:] == 0xA5)
    for a, b in zip(dev, before):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert torch.equal(out[1:-1], _call(c, [rows] * 3, q, g, dev[:4]))


def test_a_batch_without_work():
    """No rows at all, only skipped sequences, and T = 0: nothing is written."""
    c = Cache([50, 60], 1, 16, seed=116)
    q, g = (x.to(DEV) for x in rows_qg(3, 4, 117))
    dev, tab = c.device()[:4], i32(c.tables)
    out = torch.full_like(q, 3.0)
    G.kv8_decode(q, *dev, g, tab, i32([50, 60]), i32([0, 0, 0]), max_rows=2, max_kv_len=60, out=out)
    assert G.last_device_status() == 0 and torch.all(out == 3)
    G.kv8_decode(q, *dev, g, tab, i32([-1, 61]), i32([0, 2, 3]), max_rows=2, max_kv_len=60, out=out)
    assert G.last_device_status() == 6 and torch.all(out == 3)
    none = torch.empty(0, 4, 256, dtype=torch.bfloat16, device=DEV)
    assert G.kv8_decode(none, *dev, none, tab, i32([50, 60]), i32([0, 0, 0]), max_rows=1,
                        max_kv_len=60).shape == (0, 4, 256)
    k = torch.empty(0, 1, 256, dtype=torch.bfloat16, device=DEV)
    G.kv8_append(k, k, i32([]), *dev)
    G.kv8_keep(*dev, tab, i32([50, 60]), i32([0, 0, 0]), i32([]), i32([0, 0, 0]))
    assert G.last_device_status() == 0


def test_append_under_the_largest_scale():
    """A stored scale of 2^127, the largest power of two that fp32 has: the rows behind it are x 2^-127."""
    c = Cache([5, 5], 1, 16, seed=118, room=16, scale_exps=(127, 127))
    x = torch.randn(4, 1, 256, generator=torch.Generator().manual_seed(119)).bfloat16()
    x[2, 0, :9] = torch.tensor([3.3e38, -3.3e38, 1.7e38, 1e38, 3e37, 1e37, 3e36, 1e36, 1e35]).bfloat16()
    slots = [c.tables[b][0] * 16 + j for b in range(2) for j in (5, 6)]
    dev = c.device()
    G.kv8_append(x.to(DEV), x.to(DEV), i32(slots), *dev[:4])
    oracle.kv8_append(c.k, c.ks, x.double().numpy(), slots, 16)
    oracle.kv8_append(c.v, c.vs, x.double().numpy(), slots, 16)
    assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)
    assert torch.all(dev[2] == torch.from_numpy(c.ks).float().to(DEV))


def test_cache_calls_on_another_stream_and_no_allocation():
    """Plan, append and keep follow the current stream, and no call takes device memory of its own."""
    B, Hkv, bs, N = 3, 2, 16, 64
    s = torch.cuda.Stream()
    state = lambda: dict(t=i32([[-1] * 16] * B), n=i32([0] * B), f=i32(list(range(N))), c=i32([N]))  # noqa: E731
    pools = lambda: [f8(np.zeros((N, Hkv, bs, 256), np.uint8)) for _ in "kv"] + [  # noqa: E731
        torch.ones(N, Hkv, device=DEV) for _ in "kv"]
    rows = [40, 3, 20]
    src = torch.randn(63, Hkv, 256, generator=torch.Generator().manual_seed(120)).bfloat16().to(DEV)
    got = []
    for stream in (torch.cuda.current_stream(), s):
        st, pl, x = state(), pools(), torch.zeros_like(src)
        fixed = (i32([0] * B), i32(cu_of(rows)), i32([0, 7, 19, 2, 5]), i32([0, 3, 3, 5]))
        outs = torch.empty(63, dtype=torch.int32, device=DEV), torch.empty(B, dtype=torch.int32, device=DEV)
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        with torch.cuda.stream(stream):
            torch.cuda._sleep(20_000_000)               # the stream is late: x is written behind this
            x.copy_(src)
            slots, lens = G.block_plan(fixed[0], fixed[1], st["t"], st["n"], st["f"], st["c"], bs, 63,
                                       slots=outs[0], kv_lens_out=outs[1])
            G.kv8_append(x, x, slots, *pl)
            G.kv8_keep(*pl, st["t"], lens, fixed[1], fixed[2], fixed[3])
        stream.synchronize()
        if stream is s:        # (the first time round loads the kernels)
            assert torch.cuda.mem_get_info()[0] == free
        got.append([t.view(torch.uint8).clone() for t in list(st.values()) + pl])
    assert G.last_device_status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("Hq,rows", [(129, 1), (200, 1), (256, 3)])
def test_groups_wider_than_a_row_block(Hq, rows):
    c = Cache([400, rows], 1, 64, seed=121)
    q, g = rows_qg(2 * rows, Hq, 122)
    out = _call(c, [rows] * 2, q.to(DEV), g.to(DEV))
    assert_parity_dtype(out, _ref(c, [rows] * 2, q, g))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 4, 9])
def test_scales_of_zero_and_the_smallest(rows, dtype):
    """Blocks whose K scale is 0 (scores of 0), whose V scale is 0 or 2^-126, and a sequence that has
    no other: as the values say."""
    c = Cache([700, 90, 300], 2, 32, seed=123)
    t0, t1, t2 = c.tables
    c.ks[t0[2:9:3]] = 0.0
    c.vs[t0[1]], c.vs[t0[4]], c.vs[t0[5], 0] = 0.0, 2.0**-126, 0.0
    for i in range(-(-90 // 32)):
        c.vs[t1[i]] = 0.0
    for i in range(-(-300 // 32)):
        c.ks[t2[i]] = 0.0
    q, g = rows_qg(3 * rows, 12, 124, dtype)
    out, lse = _call(c, [rows] * 3, q.to(DEV), g.to(DEV), return_lse=True)
    ref = _ref(c, [rows] * 3, q, g)
    assert_parity_dtype(out, ref)
    assert torch.all(out[rows:2 * rows] == 0) and G.last_device_status() == 0
    # scores of 0: lse is ln of the keys seen, exact to an fp32 logarithm of a sum of ones
    seen = torch.arange(300 - rows + 1, 301, dtype=torch.float64)
    assert (lse[2 * rows:].double().cpu() - seen.log()[:, None]).abs().max() <= 1e-5


def test_skipped_rows_of_a_large_batch():
    """More rows than the GPU holds CTAs for: those of a skipped sequence and behind the last stay."""
    rows = [3] * 60
    c = Cache([50 + i for i in range(60)], 1, 16, seed=125)
    q, g = rows_qg(183, 16, 126)
    out = torch.full((183, 16, 256), 7.0, dtype=q.dtype, device=DEV)
    lens = list(c.lens)
    lens[20] = 2                                          # fewer keys than new rows: skipped
    G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32(lens), i32(cu_of(rows)), max_rows=3,
                 max_kv_len=max(c.lens), out=out)
    assert G.last_device_status() == 6
    assert torch.all(out[60:63] == 7) and torch.all(out[180:] == 7)
    ref = _ref(c, rows, q[:180], g[:180])
    keep = [i for i in range(180) if not 60 <= i < 63]
    assert_parity_dtype(out[keep], ref[keep])
