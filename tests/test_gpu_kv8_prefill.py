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
@pytest.mark.parametrize("rows,lens", [([1], [1]), ([100], [100]), ([5, 130, 1], [5, 700, 129]),
                                       ([127, 0, 129], [128, 40, 130]), ([64, 300], [1200, 300])])
def test_parity(rows, lens, dtype):
    c = Cache(lens, 2, 64, seed=141)
    _check(c, rows, 12, 142, dtype)
