"""Blocks that sequences share: fork, free, compact and copy, value for value against the oracle."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, codes_of, cu_of, f8, i32

pytestmark = pytest.mark.gpu


class Pool:
    """Device state of a pool beside the oracle's lists."""

    def __init__(self, B, max_blocks, N, bs, seed):
        free = torch.randperm(N, generator=torch.Generator().manual_seed(seed)).tolist()
        self.B, self.N, self.bs = B, N, bs
        self.tables = [[-1] * max_blocks for _ in range(B)]
        self.n, self.lens, self.free, self.shares = [0] * B, [0] * B, free, [0] * N
        self.d = dict(tables=i32(self.tables), n=i32(self.n), free=i32(free), fc=i32([N]), lens=i32(self.lens),
                      shares=i32(self.shares))

    def check(self):
        d, fc = self.d, self.d["fc"].item()
        assert d["tables"].tolist() == self.tables and d["n"].tolist() == self.n
        assert fc == len(self.free) and d["free"].tolist()[:fc] == self.free
        assert d["lens"].tolist() == self.lens and d["shares"].tolist() == self.shares

    def plan(self, rows):
        _, lens, served = oracle.block_plan(self.lens, rows, self.tables, self.n, self.free, self.bs, sum(rows))
        d = self.d
        _, d["lens"] = G.block_plan(d["lens"], i32(cu_of(rows)), d["tables"], d["n"], d["free"], d["fc"], self.bs,
                                    sum(rows))
        self.lens = lens
        assert G.last_device_status() == (0 if all(served) else 7)
        self.check()

    def fork(self, src, dst, lens):
        copies, verdicts = oracle.block_fork(src, dst, lens, self.lens, self.tables, self.n, self.free, self.shares,
                                             self.bs)
        d = self.d
        got = G.block_fork(i32(src), i32(dst), None if lens is None else i32(lens), d["lens"], d["tables"], d["n"],
                           d["free"], d["fc"], d["shares"], self.bs)
        assert got.tolist() == copies
        status = G.last_device_status()
        assert status in {dict(ok=0, refused=6).get(v, 7) for v in verdicts if v != "ok"} | (
            {0} if set(verdicts) <= {"ok"} else set())
        self.check()
        return got, verdicts

    def release(self, lens):
        self.lens, self.d["lens"] = list(lens), i32(lens)
        oracle.block_free(self.lens, self.tables, self.n, self.free, self.shares, self.bs)
        d = self.d
        G.block_free(d["lens"], d["tables"], d["n"], d["free"], d["fc"], d["shares"], self.bs)
        assert G.last_device_status() == 0
        self.check()

    def compact(self):
        new = oracle.block_compact(self.tables, self.n, self.free, self.shares, self.N, self.bs)
        d, before = self.d, [self.d[k].clone() for k in ("tables", "n", "free", "fc", "shares")]
        got = G.block_compact(d["tables"], d["n"], d["free"], d["fc"], d["shares"], self.bs)
        assert G.last_device_status() == 0
        for a, k in zip(before, ("tables", "n", "free", "fc", "shares")):
            assert torch.equal(a, d[k])
        assert got[0].tolist() == new[0] and got[2].tolist() == new[2] and got[3].tolist() == new[3]
        assert got[1].tolist() == list(range(self.N - 1, -1, -1))
        assert got[4].tolist() == new[4]
        self.tables, self.free, self.shares = new[0], new[1], new[2]
        d["tables"], d["free"], d["shares"] = got[:3]
        self.check()
        return got[4], new[4]


@pytest.mark.parametrize("B,bs,seed", [(4, 16, 0), (9, 64, 1), (60, 32, 2), (300, 16, 3)])
def test_rounds_of_a_server_follow_the_oracle(B, bs, seed):
    rng = np.random.RandomState(seed)
    p = Pool(B, 24, B * 12, bs, seed)
    for _ in range(6):
        # some requests end, some are cut short
        p.release([0 if rng.rand() < 0.3 else int(n * rng.choice([1, 1, 0.4])) for n in p.lens])
        # new ones behind a prefix of others
        idle = [b for b in range(B) if p.n[b] == 0]
        busy = [b for b in range(B) if p.n[b] > 0]
        rng.shuffle(idle)
        dst = idle[:len(idle) // 2] if busy else []
        src = [int(rng.choice(busy)) for _ in dst]
        lens = [int(rng.choice([0, p.lens[s], p.lens[s] // 2, p.lens[s] // bs * bs])) for s in src]
        if dst:
            p.fork(src, [int(x) for x in dst], lens)
        if rng.rand() < 0.5:
            p.compact()
        p.plan([int(rng.choice([0, 1, bs - 1, 3 * bs + 5])) if n < 18 * bs else 0 for n in p.lens])
    p.release([0] * B)
    assert sorted(p.free) == list(range(p.N)) and set(p.shares) == {0}


def test_fork_refusals_leave_the_others():
    p = Pool(8, 8, 32, 16, 5)
    p.plan([40, 16, 0, 0, 0, 5, 0, 0])
    #  ok; child holds blocks; child twice (both); longer than held; child is a parent; out of range
    _, v = p.fork([0, 0, 0, 1, 1, 5, 0, 9, 0], [2, 5, 3, 3, 4, 1, 6, 7, -1], [40, 1, 8, 8, 17, 5, 32, 3, 4])
    assert v == ["ok", "refused", "refused", "refused", "refused", "refused", "ok", "refused", "refused"]
    _, v = p.fork([0], [0], None)
    assert v == ["refused"]
    _, v = p.fork([0, 1], [3, 4], None)       # whole prefixes; the second's is one full block, shared
    assert v == ["ok", "ok"] and p.tables[4][0] == p.tables[1][0]


def test_fork_without_blocks_left():
    p = Pool(7, 4, 5, 16, 6)
    p.plan([33, 0, 0, 0, 0, 0, 0])            # three of five
    _, v = p.fork([0] * 5, [1, 2, 3, 4, 5], [33, 16, 1, 17, 32])
    assert v == ["ok", "ok", "ok", "no block", "ok"] and p.free == []
    p.release([33, 33, 0, 1, 0, 32, 0])


def test_an_empty_prefix_and_no_forks():
    p = Pool(3, 4, 6, 32, 7)
    p.plan([10, 0, 0])
    _, v = p.fork([0, 2], [1, 0], [0, 0])     # 0 is a parent and holds blocks
    assert v == ["ok", "refused"] and p.n[1] == 0
    got = G.block_fork(i32([]), i32([]), None, p.d["lens"], p.d["tables"], p.d["n"], p.d["free"], p.d["fc"],
                       p.d["shares"], p.bs)
    assert tuple(got.shape) == (0, 3)
    p.check()


def test_many_entries():
    """More than a cluster holds at once: 40 sequences of 2100 blocks, one shared by all."""
    B, W, bs = 40, 2100, 16
    N = 2 * W + B * 2
    p = Pool(B, W, N, bs, 8)
    p.plan([W * bs] + [0] * (B - 1))
    p.fork([0] * (B - 1), list(range(1, B)), [W * bs - 3 - 5 * i for i in range(B - 1)])
    # every entry but the first 20 places goes at once; 3 stays whole
    lens = [0 if b % 2 else 20 * bs for b in range(B)]
    lens[3] = p.lens[3]
    p.lens, p.d["lens"] = lens, i32(lens)
    d = p.d
    G.block_free(d["lens"], d["tables"], d["n"], d["free"], d["fc"], d["shares"], bs)
    assert G.last_device_status() == 0
    loose = []                                 # the oracle's rule, without its quadratic search
    for b, n in enumerate(lens):
        keep = min(-(-n // bs), p.n[b])
        loose += p.tables[b][keep:p.n[b]]
        p.tables[b][keep:] = [-1] * (W - keep)
        p.n[b] = keep
    last, gone = {blk: k for k, blk in enumerate(loose)}, []
    for k, blk in enumerate(loose):
        if p.shares[blk] == 0 and last[blk] == k:
            gone.append(blk)
        else:
            p.shares[blk] -= 1
    p.free += gone[::-1]
    p.check()
    p.compact()


def test_bad_states_are_recorded_and_contained():
    p = Pool(3, 4, 8, 16, 9)
    p.plan([40, 20, 0])
    d = p.d
    d["tables"][0, 1] = 77                     # outside the pool
    G.block_free(i32([0, -1, 0]), d["tables"], d["n"], d["free"], d["fc"], d["shares"], 16)
    assert G.last_device_status() == 6
    assert d["fc"].item() == 8 - 5 + 2 and d["n"].tolist() == [0, 2, 0]
    assert d["tables"][0].tolist() == [-1] * 4 and d["tables"][1].tolist() == p.tables[1]
    # a stack that holds a block twice: nothing moves
    free = i32([4, 4, 5, 0, 0, 0, 0, 0])
    got = G.block_compact(d["tables"], d["n"], free, i32([3]), d["shares"], 16)
    assert G.last_device_status() == 6
    assert got[4].tolist() == [[-1, -1, 0]] * 4 and torch.equal(got[1], free)
    # a table that names a free block
    n, tables = i32([2]), i32([[1, 3, -1]])
    got = G.block_compact(tables, n, i32([3, 0, 2, 0]), i32([3]), i32([0] * 4), 16)
    assert G.last_device_status() == 6
    assert got[0].tolist() == [[0, -1, -1]] and got[3].tolist() == [-1, 0, -1, -1]


@pytest.mark.parametrize("Hkv,bs,n", [(1, 16, 3), (2, 128, 9), (5, 64, 40), (4, 16, 700)])
def test_copy_is_bit_exact(Hkv, bs, n):
    rng = np.random.RandomState(n)
    N = 2 * n + 3
    pools = [rng.randint(0, 256, (N, Hkv, bs, 256)).astype(np.uint8) for _ in "kv"]
    scales = [rng.rand(N, Hkv).astype(np.float32) for _ in "kv"]
    perm = rng.permutation(N)
    copies = [[int(perm[2 * i]), int(perm[2 * i + 1]), int(rng.choice([1, bs - 1, bs, 7]))] for i in range(n)]
    for i in range(0, n, 3):
        copies[i] = [-1, copies[i][1], 5] if i % 2 else [copies[i][0], copies[i][1], 0]
    dev = [f8(p) for p in pools], [torch.from_numpy(s).to(DEV) for s in scales]
    G.kv8_copy(i32(copies), *dev[0], *dev[1])
    assert G.last_device_status() == 0
    oracle.kv8_copy(copies, pools, scales)
    for a, b in zip(dev[0], pools):
        assert np.array_equal(codes_of(a), b)
    for a, b in zip(dev[1], scales):
        assert np.array_equal(a.cpu().numpy(), b)


def test_copies_out_of_range_are_skipped():
    pools = [f8(np.zeros((4, 1, 16, 256), np.uint8)) for _ in "kv"]
    scales = [torch.arange(4, dtype=torch.float32, device=DEV)[:, None] for _ in "kv"]
    scales = [s.contiguous() for s in scales]
    G.kv8_copy(i32([[0, 4, 3], [7, 1, 3], [2, 3, 17], [1, 1, 16], [0, 2, 1]]), *pools, *scales)
    assert G.last_device_status() == 6
    assert scales[0].flatten().tolist() == [0, 1, 0, 3]
    G.kv8_copy(i32(np.zeros((0, 3)).tolist()).reshape(0, 3), *pools, *scales)


def test_captured_fork_and_free_replay():
    """A graph of a fork, its copy and the free of the child gives the pool back each time."""
    p = Pool(2, 4, 8, 16, 10)
    p.plan([37, 0])
    d = p.d
    pools = [f8(np.random.RandomState(1).randint(0, 120, (8, 2, 16, 256)).astype(np.uint8)) for _ in "kv"]
    scales = [torch.rand(8, 2, device=DEV) for _ in "kv"]
    src, dst, ended, copies = i32([0]), i32([1]), i32([37, 0]), torch.empty(1, 3, dtype=torch.int32, device=DEV)

    def step():
        G.block_fork(src, dst, None, d["lens"], d["tables"], d["n"], d["free"], d["fc"], d["shares"], 16, copies=copies)
        G.kv8_copy(copies, *pools, *scales)
        G.block_free(ended, d["tables"], d["n"], d["free"], d["fc"], d["shares"], 16)

    step()
    torch.cuda.synchronize()
    state = {k: v.clone() for k, v in d.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert G.last_device_status() == 0
    for k, v in state.items():
        assert torch.equal(v, d[k])
    a, b, rows = copies[0].tolist()
    assert rows == 5 and np.array_equal(codes_of(pools[0])[b, :, :5], codes_of(pools[0])[a, :, :5])
