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
