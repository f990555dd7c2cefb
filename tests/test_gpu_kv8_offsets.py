"""Block planning where row offsets fall: a sequence that is served has a slot for each of its rows."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
from tests.kv8_cases import DEV, i32

pytestmark = pytest.mark.gpu


def _plan(lens, cu, have, max_blocks, N, bs, T):
    """What block_plan() has to give: a sequence is served when it keeps the bounds, its rows start at or
    behind the end of every earlier one that keeps them, and its blocks fit.  Returns tables, n_blocks,
    free list, slots, lengths; `have`: blocks owned, handed out in order from the bottom of the pool."""
    B = len(lens)
    tables, at = [], 0
    for n in have:
        m = min(n, max_blocks)
        tables.append(list(range(at, at + m)) + [-1] * (max_blocks - m))
        at += m
    free = list(range(at, N))
    start = [list(t) for t in tables], list(free)
    end, ok = 0, []
    for b in range(B):
        own = (lens[b] >= 0 and 0 <= cu[b] <= cu[b + 1] <= T and 0 <= have[b] <= max_blocks
               and lens[b] + cu[b + 1] - cu[b] <= max_blocks * bs)
        ok.append(own and cu[b] >= end)
        if own:
            end = max(end, cu[b + 1])
    n_blocks, out, slots = list(have), list(lens), [-1] * T
    loose = []
    need = [-(-(lens[b] + cu[b + 1] - cu[b]) // bs) if ok[b] else 0 for b in range(B)]
    for b in range(B):
        if ok[b] and need[b] < have[b]:
            loose += tables[b][need[b]:have[b]]
            tables[b][need[b]:have[b]] = [-1] * (have[b] - need[b])
            n_blocks[b] = need[b]
    free += loose[::-1]
    left, wanted = len(free), 0
    for b in range(B):
        if not ok[b]:
            continue
        grow = need[b] - n_blocks[b]
        wanted += grow
        if grow == 0 or wanted <= left:
            for i in range(n_blocks[b], need[b]):
                tables[b][i] = free.pop()
            n_blocks[b], out[b] = need[b], lens[b] + cu[b + 1] - cu[b]
            for i in range(cu[b + 1] - cu[b]):
                pos = lens[b] + i
                slots[cu[b] + i] = tables[b][pos // bs] * bs + pos % bs
    return start, tables, n_blocks, free, slots, out, all(ok)


def _check(lens, cu, have, max_blocks, N, bs, T):
    (t0, f0), tables, n_blocks, free, slots, out, fine = _plan(lens, cu, have, max_blocks, N, bs, T)
    d = dict(t=i32(t0), n=i32(have), f=i32(f0 + [0] * (N - len(f0))), c=i32([len(f0)]))
    got, lo = G.block_plan(i32(lens), i32(cu), d["t"], d["n"], d["f"], d["c"], bs, T)
    assert G.last_device_status() == (0 if fine else 6)
    assert lo.tolist() == out and d["n"].tolist() == n_blocks
    assert d["t"].tolist() == tables and d["c"].item() == len(free)
    assert d["f"].tolist()[:len(free)] == free
    assert got.tolist() == slots


@pytest.mark.parametrize("lens,cu,have", [
    ([0, 0, 0, 0, 0], [0, 1, 2, 3, 2, 4], [0, 0, 3, 0, 0]),     # the one before the fall is out of bounds itself
    ([-1, 32, 0, 0, 0], [0, 1, 2, 3, 2, 4], [0, 0, 3, 0, 0]),
    ([0, 0, 0], [0, 4, 2, 6], [0, 0, 0]),                       # rows that an earlier sequence has
    ([0, 5, 9, 3], [0, 4, 2, 4, 6], [0, 1, 1, 1]),              # the next but one may go on
    ([0, 5, 9, 3], [0, 6, 5, 6, 6], [0, 1, 1, 1]),
    ([0, 0, 3, 9], [3, 2, 2, 3, 4], [0, 0, 1, 1]),
    ([0, 0, 0], [0, -1, 2, 3], [0, 0, 0]),
    ([7, 7, 7, 7], [0, 0, 0, 0, 0], [1, 2, 0, 1]),
])
def test_rows_after_offsets_that_fall(lens, cu, have):
    _check(lens, cu, have, 2, 20, 16, 7)


@pytest.mark.parametrize("B,T", [(60, 400), (1500, 9000), (3000, 2000)])
def test_random_offsets(B, T):
    """One CTA, and a cluster of eight: a few falls among many sequences."""
    rng = np.random.RandomState(B)
    for falls in (0, 1, 7):
        cu = np.sort(rng.randint(0, T + 1, B + 1))
        for i in rng.randint(1, B, falls):
            cu[i] = rng.randint(-2, T + 3)
        lens = rng.randint(0, 40, B)
        lens[rng.randint(0, B, 3)] = -1
        have = rng.randint(0, 4, B).tolist()
        _check(lens.tolist(), cu.tolist(), have, 8, 9 * B, 16, T)
