"""Attention over the paged 8-bit cache against an error bound of every element's own."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
from tests.kv8_cases import DEV, Cache, cu_of, i32, rows_qg
from tests.parity import to_f64

pytestmark = pytest.mark.gpu

U = {torch.bfloat16: 2.0**-8, torch.float16: 2.0**-11}


def _bounded(c, rows, Hq, seed, dtype):
    """Chain rows of one sequence.  With s the scores, w the probabilities and A = sum w |v| sigmoid(g),
    an output may be off by

        A (2 ds + 2 u + 2^-13) + F + 2^-25
                                  u: half a step of the type, for P's terms and for the output;
                                    sums of weights in fp32; fp16's smallest half step
        ds <= (2^-16 sum |q k| + 2^-19 max |q| sum |k|) ks / 16   256 fp32 sums, and what the terms
                                    of a row's small elements of Q lose, the largest over its keys
        F = n 2^-24 max(w vs) 448   the probabilities' own step, with the values' scale, 2^-24 of the
                                    largest; a code is 448 at most
    """
    (n,) = c.lens
    q, g = rows_qg(rows, Hq, seed, dtype)
    out, lse = G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32(c.lens),
                            i32(cu_of([rows])), max_rows=rows, max_kv_len=n, return_lse=True)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    blocks = [c.tables[0][j // c.bs] for j in range(n)]
    qq, gg, got, gl = to_f64(q), to_f64(g), to_f64(out), to_f64(lse)
    gqa = Hq // c.Hkv
    for t in range(rows):
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
            tol = (w @ np.abs(vv)) * sig * (2 * ds + 2 * U[dtype] + 2.0**-13)
            tol += m * 2.0**-24 * (w * vs).max() * 448 + 2.0**-25
            err = np.abs(got[t, h] - (w @ vv) * sig)
            assert np.all(err <= tol), (t, h, (err / tol).max())
            assert abs(gl[t, h] - (s.max() + np.log(l))) <= ds + 1e-5


@pytest.mark.parametrize("rows", [1, 3, 5, 9])       # 4, 12, 20 and 36 packed rows
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block_scales_far_apart(dtype, rows):
    """A block of tiny values that takes nearly all probability next to large ones, and keys whose scores
    differ by tens."""
    c = Cache([400], 2, 16, seed=59)
    for i, e in enumerate([-60, -7, 3, -30, -7, -20, -7, 0]):
        c.vs[c.tables[0][i]] = 2.0 ** e
        c.ks[c.tables[0][i]] = 2.0 ** [-7, -30, -7, -3, -7, -9, -40, -7][i]
    _bounded(c, rows, 8, 60, dtype)


@pytest.mark.parametrize("rows", [1, 3, 5, 9])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_block_scales_that_move_both_references(dtype, rows):
    """V's scales fall and rise by 2^20 and more from tile to tile, K's by 16."""
    c = Cache([3000], 2, 64, seed=171)
    rng = np.random.RandomState(172)
    for i in range(-(-3000 // 64)):
        c.vs[c.tables[0][i]] = 2.0 ** (-6 + rng.randint(-14, 15))
        c.ks[c.tables[0][i]] = 2.0 ** (-7 + rng.randint(-2, 3))
    _bounded(c, rows, 8, 173, dtype)


@pytest.mark.parametrize("rows", [1, 3, 9])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_ordinary_blocks(dtype, rows):
    _bounded(Cache([2500], 2, 32, seed=174), rows, 8, 175, dtype)


def test_workspace_holds_every_row_in_its_parts():
    """Three parts of 256 values and a sum for each row at least, in fp32; sixteen sequences take sixteen
    times the rows of one."""
    for B, Hq, Hkv, n in [(1, 24, 4, 512), (16, 24, 4, 32768), (64, 16, 2, 1500)]:
        assert G.kv8_workspace_size(B, B, Hq, Hkv, 1, n) >= B * Hq * 257 * 4 * 3
