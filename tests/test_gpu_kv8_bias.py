"""The rounding of the probabilities' terms leaves no share of V over on the whole."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, cu_of, i32
from tests.parity import to_f64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 3, 4, 16])          # 8, 24, 32 and 128 packed rows
def test_outputs_are_not_too_large_on_the_whole(rows, dtype):
    """V's values are positive, 0.5 to 1.5, and outputs about 1 times their gates, which spread them
    smoothly over the type's steps.  An output's rounding is off by 2^-8 of it (fp16 2^-11) at most,
    either way alike, 2^-8 / sqrt(3) in the mean square; a row's terms are off by as much for each
    of the hundreds of keys that share its weight, alike for its 256 values.  So the mean over n
    values of r rows is within 5 deviations of 0 when below
        5 * 2^-8 / sqrt(3) * (1 / sqrt(n) + 1 / sqrt(100 r))."""
    n, Hq, B = 3000, 8, 24
    c = Cache([n] * B, 1, 64, seed=180)
    gen = torch.Generator().manual_seed(181)
    c.v[:] = oracle.e4m3_encode((32 + 64 * torch.rand(c.v.shape, generator=gen)).double().numpy())
    c.vs[:] = 2.0**-6
    c.ks[:] = 2.0**-6
    q, g = (torch.randn(B * rows, Hq, 256, generator=gen).to(dtype) for _ in range(2))
    out = G.kv8_decode(q.to(DEV), *c.device()[:4], g.to(DEV), i32(c.tables), i32(c.lens),
                       i32(cu_of([rows] * B)), max_rows=rows, max_kv_len=n)
    assert G.last_device_status() == 0
    k, v = c.contiguous()
    ref = oracle.decode(to_f64(q), k, v, to_f64(g), c.lens, cu_of([rows] * B))[0]
    mean = (to_f64(out) / ref - 1).mean()
    half = 2.0**-8 if dtype == torch.bfloat16 else 2.0**-11
    assert abs(mean) <= 5 * half / 3**0.5 * (ref.size**-0.5 + (100 * B * rows * Hq) ** -0.5)
