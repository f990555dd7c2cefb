"""Prompt chunks and copies of blocks behind the 2^32-byte mark of a pool: the bits that the same blocks of a small pool
give."""
import pytest
import torch

import gqa_head_gated_gb300 as G
from tests.kv8_cases import DEV, Cache, cu_of, i32, rows_qg

pytestmark = pytest.mark.gpu

HKV, BS, N = 2, 64, 160000          # 5.2e9 bytes each of K and V


@pytest.fixture(scope="module")
def pools():
    """A small pool and a large one whose last blocks are the small one's."""
    c = Cache([900, 77, 300], HKV, BS, seed=230, room=40, spare=6)
    small = c.device()
    big = [torch.zeros(N, HKV, BS, 256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in "kv"]
    big += [torch.ones(N, HKV, device=DEV) for _ in "kv"]
    at = N - c.N
    assert at * HKV * BS * 256 > 1 << 32
    for b, s in zip(big, small):
        b[at:].view(torch.uint8).copy_(s.view(torch.uint8))
    yield c, small, big, at


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_chunks(pools, dtype):
    c, small, big, at = pools
    rows = [200, 77, 9]
    q, g = (x.to(DEV) for x in rows_qg(sum(rows), 8, 231, dtype))
    tables = torch.where(small[4] >= 0, small[4] + at, small[4])
    a, la = G.kv8_prefill(q, *small[:4], g, small[4], i32(c.lens), i32(cu_of(rows)), return_lse=True)
    b, lb = G.kv8_prefill(q, *big, g, tables, i32(c.lens), i32(cu_of(rows)), return_lse=True)
    assert G.last_device_status() == 0
    assert torch.equal(a, b) and torch.equal(la, lb) and not torch.isnan(a.float()).any()


def test_copies(pools):
    """From behind the mark to before it and back to another place behind it, and rows of a block alone."""
    c, small, big, at = pools
    a, b, spare = c.tables[0][0], c.tables[0][3], sorted(set(range(c.N)) - {t for row in c.tables for t in row})
    x, y = spare[:2]
    G.kv8_copy(i32([[at + a, 5, BS], [at + b, 131071, 23]]), *big)
    G.kv8_copy(i32([[5, at + x, BS], [131071, at + y, 23], [5, N, 3]]), *big)
    assert G.last_device_status() == 6                  # N is no block
    for big_t, small_t in zip(big, small):
        s, d = small_t.view(torch.uint8), big_t.view(torch.uint8)
        assert torch.equal(d[at + x], s[a]) and torch.equal(d[5], s[a])
        if s.dim() == 4:
            assert torch.equal(d[at + y, :, :23], s[b, :, :23]) and torch.equal(d[at + y, :, 23:], s[y, :, 23:])
            assert torch.equal(d[131071, :, :23], s[b, :, :23]) and not d[131071, :, 23:].any()
        else:
            assert torch.equal(d[at + y], s[b])
        rest = [n for n in range(c.N) if n not in (x, y)]
        assert torch.equal(d[at:][rest], s[rest])
        assert not d[:5].view(torch.int64).any() or s.dim() == 2
