"""Outputs of rope whose rows share memory are refused before a launch."""
import ctypes
import os

import pytest

from gqa_head_gated_gb300 import _lib

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from gqa_head_gated_gb300 import build
        build.build()
    return _lib.load()


def _codes(lib, q_out, B, L, Hq, k_out=None, Hkv=0):
    """Both types' codes for outputs of these strides (batch, token, head)."""
    dense = [L * Hq * 256, Hq * 256, 256]
    s = (ctypes.c_longlong * 12)(*dense, *q_out, *([L * Hkv * 256, Hkv * 256, 256] + k_out if k_out else [0] * 6))
    return [f(P(16), P(32) if k_out else None, P(48), P(64), P(80), P(96) if k_out else None, s, B, L, Hq, Hkv, 64, 0, 0,
              0, 1.0, None) for f in (lib.gqa_rope, lib.gqa_rope_f16)]


@pytest.mark.parametrize("B,L,Hq,strides", [
    (1, 3, 4, [0, 256, 256]),              # tokens on heads
    (1, 3, 4, [0, 512, 256]), (1, 3, 4, [0, 768, 256]),
    (1, 3, 4, [0, 256, 512]), (2, 3, 4, [256, 1024, 256]), (2, 3, 4, [1024, 1024, 256]),
    (2, 3, 4, [2048, 1024, 256]),          # the second entry on the first's third token
    (2, 5, 1, [1024, 264, 0]),             # rows that overlap in part: 4 * 264 = 1056
    (3, 3, 1, [776, 512, 0]),              # 776 and 1024 are 248 apart
    (1, 2, 1 << 19, [0, (1 << 19) * 256 - 256, 256]),
])
def test_rows_that_overlap_are_refused(lib, B, L, Hq, strides):
    assert _codes(lib, strides, B, L, Hq) == [1, 1]


def test_k_out_is_checked_too(lib):
    assert _codes(lib, [0, 1024, 256], 1, 3, 4, [0, 256, 256], 2) == [1, 1]

