"""The ramp of "yarn" where its two ends fall together: pairs below beta_slow turns go over, those above beta_fast stay."""
import math

import pytest
import torch

import gqa_head_gated_gb300 as G


@pytest.mark.parametrize("original_len,beta_fast,beta_slow", [(4, 32.0, 1.0), (6, 32.0, 1.0), (4096, 1000.0, 700.0),
                                                               (4096, 1e6, 652.0), (10 ** 9, 3.0, 1.0), (10 ** 15, 32.0, 1.0),
                                                               (4096, 32.0, 1.0), (100, 32.0, 1.0), (32768, 1.01, 1.0)])
def test_yarn_at_its_ends(original_len, beta_fast, beta_slow):
    rot, base, factor = 64, 1e4, 4.0
    f, _ = G.rope_frequencies(rot, base, device="cpu")
    g, _ = G.rope_frequencies(rot, base, "yarn", factor, original_len, beta_fast, beta_slow, device="cpu")
    turns = original_len * base ** (-2.0 * torch.arange(rot // 2, dtype=torch.float64) / rot) / (2 * math.pi)
    step = base ** (2.0 / rot)      # the ends of the ramp are whole pairs, each up to a pair outside
    # (both in 64 bits, rounded once: half a step each)
    slow, fast = turns < beta_slow / step * (1 - 1e-9), turns > beta_fast * step * (1 + 1e-9)
    if original_len * 1.0 / (2 * math.pi) < beta_slow:
        slow = turns < beta_slow
    assert torch.equal(g[fast], f[fast])
    assert torch.allclose(g[slow], f[slow] / factor, rtol=2.0 ** -23, atol=0)
    assert slow.any() or fast.any()
    assert ((g <= f) & (g >= f / factor * (1 - 2.0 ** -23))).all()
