"""Rotary positions of views whose dims of one have strides of their own, as torch leaves them."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
from tests.kv8_cases import DEV, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stride", [1, 3, 0, 1020, 2 ** 40 + 1])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_dims_of_one_with_any_stride(stride, dtype):
    f, _ = G.rope_frequencies(64)
    x = torch.randn(6, 256, generator=torch.Generator().manual_seed(1)).to(DEV, dtype)
    # one token of six heads, six tokens of one head, one of each; and one head of [B, H, L, 256]
    token, head, both = (x.as_strided(*a) for a in (((1, 6, 256), (stride, 256, 1)), ((6, 1, 256), (256, stride, 1)),
                                                    ((1, 1, 256), (stride, stride, 1))))
    heads = x.as_strided((2, 1, 3, 256), (3 * 256, stride, 256, 1))
    for t, p in ((token, [9]), (head, [1, 2, 3, 4, 5, 6]), (both, [9])):
        want, _ = G.rope(torch.empty(t.shape, dtype=dtype, device=DEV).copy_(t), None, i32(p), f)
        got, k = G.rope(t, t, i32(p), f)
        assert torch.equal(got, want) and torch.equal(k, want)
        y = x.clone()
        z = y.as_strided(t.shape, t.stride())
        G.rope(z, None, i32(p), f, q_out=z)
        assert torch.equal(z, want)
    want, _ = G.rope(torch.empty(heads.shape, dtype=dtype, device=DEV).copy_(heads), None, i32([5, 6, 7]), f)
    assert torch.equal(G.rope(heads, None, i32([5, 6, 7]), f)[0], want)
    assert G.last_device_status() == 0


def test_outputs_of_any_strides_whose_rows_lie_apart():
    """Against all pairs of rows: outputs with overlapping rows are refused, all others are written in place and
    nothing beside them."""
    rng = np.random.RandomState(3)
    T, H = 3, 3
    f, _ = G.rope_frequencies(64)
    q, p = torch.randn(T, H, 256, generator=torch.Generator().manual_seed(2)).to(DEV, torch.bfloat16), i32(list(range(T)))
    want, _ = G.rope(q, None, p, f)
    seen = [0, 0]
    for _ in range(300):
        token, head = (8 * int(rng.randint(32, 200)) for _ in "th")
        at = sorted(t * token + h * head for t in range(T) for h in range(H))
        apart = all(b - a >= 256 for a, b in zip(at, at[1:]))
        mem = torch.full((at[-1] + 256,), 5.0, dtype=torch.bfloat16, device=DEV)
        out = mem.as_strided((T, H, 256), (token, head, 1))
        seen[apart] += 1
        if not apart:
            with pytest.raises(G.GqaError):
                G.rope(q, None, p, f, q_out=out)
            continue
        G.rope(q, None, p, f, q_out=out)
        assert torch.equal(out, want)
        out.fill_(5.0)
        assert torch.all(mem == 5)
    assert min(seen) > 20 and G.last_device_status() == 0
