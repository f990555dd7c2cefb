"""Chunks of very many short sequences: shares of one-tile segments, of which the odd CTA of a pair has no key to
bring (64 keys and fewer) beside ones of which it has."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, cu_of, i32, rows_qg
from tests.parity import assert_parity_dtype, to_f64
from tests.test_gpu_kv8_decode import LSE_TOL

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens", [[64], [1, 33, 64, 17], [20, 64, 65, 40, 3, 128, 50, 9, 64, 200, 60], [64, 192, 30, 320]])
def test_shares_of_short_segments(lens, dtype):
    """200 sequences x 4 KV heads: some ten segments a pair.  The same bits each time, and no wait runs out."""
    B, Hkv, Hq = 200, 4, 8
    lens = (lens * B)[:B]
    c = Cache(lens, Hkv, 16, seed=211)
    rows = [min(n, 1 + b % 5) for b, n in enumerate(lens)]
    q, g = (x.to(DEV) for x in rows_qg(sum(rows), Hq, 212, dtype))
    dev, tables, kv, cu = c.device()[:4], i32(c.tables), i32(lens), i32(cu_of(rows))
    ws = torch.empty(G.kv8_prefill_workspace_size(), dtype=torch.uint8, device=DEV)

    def call():
        return G.kv8_prefill(q, *dev, g, tables, kv, cu, max_rows=5, max_kv_len=max(lens), workspace=ws,
                             return_lse=True)

    out, lse = call()
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    ref, rl = oracle.decode(to_f64(q), k, v, to_f64(g), lens, cu_of(rows))
    assert_parity_dtype(out, ref)
    assert np.abs(to_f64(lse) - rl).max() <= LSE_TOL
    differ = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(300):
        again, _ = call()
        differ += (again != out).sum()
    assert G.last_device_status() == 0 and differ.item() == 0
