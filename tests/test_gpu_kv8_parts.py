"""A key with NaN values that a row sees gives NaN, whichever part of the sequence it falls in."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, cu_of, i32, rows_qg
from tests.parity import assert_nonfinite_parity, to_f64

pytestmark = pytest.mark.gpu


# 8 and 64 packed rows (a CTA merges a row), and 60 sequences (a group of threads a row)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,rows,Hq,n", [(1, 1, 8, 4000), (1, 8, 8, 4000), (60, 2, 16, 1500), (60, 5, 8, 1500)])
def test_nan_values_of_a_key_far_below_the_others(B, rows, Hq, n, dtype):
    """Key 3 stands 208 nats above the rest (their weights beside its are 0 in fp32), the last key's
    and one middle key's V hold NaN: it shows in their dims, and only there."""
    c = Cache([n] * B, 1, 64, seed=160)
    q, g = rows_qg(B * rows, Hq, 161, dtype)
    q[:, :, 0] = 16.0
    for b in range(B):
        for j in range(n):
            c.k[c.tables[b][j // 64], 0, j % 64, 0] = 0
        c.k[c.tables[b][0], 0, 3, 0] = int(oracle.e4m3_encode(np.array([208.0]))[0])
        c.ks[c.tables[b][0]] = 1.0
        c.k[c.tables[b][0], 0, :, 1:] = 0
        for j, d in ((n // 2, 7), (n - rows, 200)):
            c.v[c.tables[b][j // 64], 0, j % 64, d] = 0x7F
    out = G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32(c.lens),
                       i32(cu_of([rows] * B)), max_rows=rows, max_kv_len=n)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    with np.errstate(all="ignore"):
        ref = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, cu_of([rows] * B))[0]
    assert np.isnan(ref[..., [7, 200]]).all() and np.isnan(ref).mean() == 2 / 256
    assert_nonfinite_parity(out, ref)
