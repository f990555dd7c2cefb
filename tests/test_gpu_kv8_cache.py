"""Block planning, quantising append and keep of the paged 8-bit cache, value for value
against the oracle."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, codes_of, cu_of, f8, i32

pytestmark = pytest.mark.gpu


class Planner:
    """Device state of a pool beside the oracle's lists."""

    def __init__(self, B, max_blocks, N, bs, seed):
        free = torch.randperm(N, generator=torch.Generator().manual_seed(seed)).tolist()
        self.bs, self.B = bs, B
        self.o = dict(tables=[[-1] * max_blocks for _ in range(B)], n=[0] * B, free=free, lens=[0] * B)
        self.d = dict(tables=i32(self.o["tables"]), n=i32([0] * B), free=i32(free), fc=i32([N]),
                      lens=i32([0] * B))

    def step(self, rows, pad=0, in_place=False):
        T = sum(rows) + pad
        slots, lens, served = oracle.block_plan(self.o["lens"], rows, self.o["tables"], self.o["n"],
                                                self.o["free"], self.bs, T)
        d = self.d
        got, out = G.block_plan(d["lens"], i32(cu_of(rows)), d["tables"], d["n"], d["free"], d["fc"],
                                self.bs, T, kv_lens_out=d["lens"] if in_place else None)
        assert got.tolist() == slots and out.tolist() == lens
        assert d["tables"].tolist() == self.o["tables"] and d["n"].tolist() == self.o["n"]
        fc = d["fc"].item()
        assert fc == len(self.o["free"]) and d["free"].tolist()[:fc] == self.o["free"]
        assert G.last_device_status() == (0 if all(served) else 7)
        self.o["lens"], self.d["lens"] = lens, out
        return served

    def set_lens(self, lens):
        self.o["lens"], self.d["lens"] = list(lens), i32(lens)


@pytest.mark.parametrize("B,bs,seed", [(1, 16, 0), (3, 64, 1), (37, 32, 2), (700, 128, 3)])
def test_plan_steps_follow_the_oracle(B, bs, seed):
    rng = np.random.RandomState(seed)
    p = Planner(B, 40, B * 24, bs, seed)
    for step in range(8):
        rows = rng.choice([0, 1, 1, 2, bs - 1, bs, bs + 1, 3 * bs + 5], B).tolist()
        room = 40 * bs
        rows = [r if n + r <= room else 0 for n, r in zip(p.o["lens"], rows)]
        p.step(rows, pad=int(rng.randint(0, 5)), in_place=bool(step & 1))
        # some requests end, some drafts are refused
        cut = [0 if rng.rand() < 0.2 else max(0, n - int(rng.randint(0, 3))) for n in p.o["lens"]]
        p.set_lens(cut)
    p.set_lens([0] * B)
    p.step([0] * B)                       # everything is given back
    assert p.d["fc"].item() == B * 24
    assert sorted(p.d["free"].tolist()) == list(range(B * 24))


def test_plan_first_come_first_served_when_blocks_run_out():
    p = Planner(4, 8, 6, 16, 5)
    assert p.step([40, 33, 17, 0], pad=2) == [True, True, False, True]    # 3 + 3 of 6, then 2 more
    assert p.step([8, 1, 1, 0]) == [True, True, False, True]   # room in blocks they own
    p.set_lens([0] + p.o["lens"][1:])
    assert p.step([0, 1, 17, 1]) == [True, True, True, True]


def test_plan_refuses_sequences_that_break_the_bounds():
    B, bs, N = 5, 16, 20
    tables = [[-1] * 2 for _ in range(B)]
    d = dict(tables=i32(tables), n=i32([0, 0, 3, 0, 0]), free=i32(list(range(N))), fc=i32([N]))
    # -1 keys; 33 keys in two blocks; owns three of two; falls; fine
    lens = i32([-1, 32, 0, 0, 0])
    slots, out = G.block_plan(lens, i32([0, 1, 2, 3, 2, 4]), d["tables"], d["n"], d["free"], d["fc"],
                              bs, 5)
    assert G.last_device_status() == 6
    assert out.tolist() == [-1, 32, 0, 0, 2]
    assert d["n"].tolist() == [0, 0, 3, 0, 1] and d["fc"].item() == N - 1
    assert slots.tolist()[:2] == [-1, -1] and slots.tolist()[4] == -1
    assert d["tables"].tolist()[:4] == tables[:4] and d["tables"].tolist()[4] == [N - 1, -1]
    # a stack higher than its list: bounded, recorded
    fc = i32([N + 7])
    G.block_plan(i32([0]), i32([0, 16]), i32([[-1]]), i32([0]), d["free"], fc, bs, 16)
    assert G.last_device_status() == 6 and fc.item() == N - 1


def test_plan_most_sequences():
    B = 8192
    p = Planner(B, 1, B, 16, 6)
    p.step([1] * B)
    p.step([0] * B)
    with pytest.raises(G.GqaError) as e:
        G.block_plan(i32([0] * (B + 1)), i32([0] * (B + 2)), i32([[-1]] * (B + 1)), i32([0] * (B + 1)),
                     i32([0]), i32([0]), 16, 0)
    assert e.value.code == 2


# ------------------------------------------------------------------------------- append

def _append(c, x, y, slots):
    """Appends on both sides; every code and scale of the pools has to be the same."""
    dev = c.device()
    G.kv8_append(x.to(DEV), y.to(DEV), i32(slots), *dev[:4])
    status = G.last_device_status()
    oracle.kv8_append(c.k, c.ks, x.double().numpy(), slots, c.bs)
    oracle.kv8_append(c.v, c.vs, y.double().numpy(), slots, c.bs)
    for t, codes in zip(dev[:2], (c.k, c.v)):
        assert np.array_equal(codes_of(t), codes)
    for t, s in zip(dev[2:4], (c.ks, c.vs)):
        assert np.array_equal(t.double().cpu().numpy(), s)
    return status


def _new(T, Hkv, seed, dtype, spread=0.0):
    gen = torch.Generator().manual_seed(seed)
    one = lambda: (torch.randn(T, Hkv, 256, generator=gen)  # noqa: E731
                   * torch.exp2(torch.randn(T, 1, 1, generator=gen) * spread)).to(dtype)
    return one(), one()


def _slots(c, b, start, n):
    return [c.tables[b][j // c.bs] * c.bs + j % c.bs for j in range(start, start + n)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("rows", [[1, 1, 1], [5, 0, 130], [64, 63, 65], [300, 1, 17]])
def test_append_value_for_value(rows, bs, dtype):
    held = [7, 64, 0]
    c = Cache(held, 3, bs, seed=11, room=300)
    slots = sum((_slots(c, b, held[b], r) for b, r in enumerate(rows)), [])
    # runs whose scales grow over what their blocks hold, and runs whose do not
    x, y = _new(sum(rows), 3, 12, dtype, spread=3.0)
    assert _append(c, x, y, slots) == 0


def test_append_one_head_long_prompt_and_skipped_rows():
    c = Cache([0, 3], 1, 64, seed=13, room=1000)
    slots = _slots(c, 0, 0, 700) + [-1] * 9 + _slots(c, 1, 3, 291) + [-1]
    x, y = _new(len(slots), 1, 14, torch.bfloat16)
    assert _append(c, x, y, slots) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_append_extreme_values(dtype):
    """Zeros, the type's largest, smallest and subnormal values, NaN and infinities."""
    info = torch.finfo(dtype)
    vals = [0.0, info.max, info.tiny, info.smallest_normal / 64, -info.max, 448.0, 449.0, 1.0,
            float("nan"), float("inf"), -float("inf"), -0.0]
    c = Cache([0] * len(vals), 2, 16, seed=15, room=16)
    x, y = _new(2 * len(vals), 2, 16, dtype)
    for i, v in enumerate(vals):
        x[2 * i] = v                 # a row of nothing else, then an ordinary one behind it
        y[2 * i, :, 5] = v
    slots = sum((_slots(c, b, 0, 2) for b in range(len(vals))), [])
    assert _append(c, x, y, slots) == 0
    # and each behind rows that its block holds
    c = Cache([5] * len(vals), 2, 16, seed=17, room=16)
    slots = sum((_slots(c, b, 5, 2) for b in range(len(vals))), [])
    assert _append(c, x, y, slots) == 0


def test_append_twice_is_appending_behind():
    """Rows in one call, and one by one: the same scales, and codes that differ only where a
    value was rounded more than once."""
    a, b = Cache([0], 2, 32, seed=18, room=64), Cache([0], 2, 32, seed=18, room=64)
    x, y = _new(40, 2, 19, torch.bfloat16, spread=2.0)
    assert _append(a, x, y, _slots(a, 0, 0, 40)) == 0
    for i in range(40):
        assert _append(b, x[i:i + 1], y[i:i + 1], _slots(b, 0, i, 1)) == 0
    assert np.array_equal(a.ks, b.ks) and np.array_equal(a.vs, b.vs)


def test_append_skips_bad_slots():
    c = Cache([0, 0], 1, 16, seed=20, room=32)
    k0, v0 = c.k.copy(), c.v.copy()
    dev = c.device()
    x, y = _new(6, 1, 21, torch.bfloat16)
    n = c.N * 16
    s = _slots(c, 0, 0, 3)
    # past the pool, far below, the same place twice, and a row behind that one
    G.kv8_append(x.to(DEV), y.to(DEV), i32([n, -5, s[0], s[0], s[0] + 1, -1]), *dev[:4])
    assert G.last_device_status() == 6
    oracle.kv8_append(c.k, c.ks, x[2:3].double().numpy(), [s[0]], 16)
    oracle.kv8_append(c.v, c.vs, y[2:3].double().numpy(), [s[0]], 16)
    assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)
    assert not np.array_equal(k0, c.k)


# ------------------------------------------------------------------------------- keep

def _keep(c, rows, keep):
    dev = c.device()
    out = torch.full((len(rows),), -9, dtype=torch.int32, device=DEV)
    flat = [i for k in keep for i in k]
    G.kv8_keep(*dev, i32(c.lens), i32(cu_of(rows)), i32(flat), i32(cu_of([len(k) for k in keep])), out)
    return dev, out.tolist(), G.last_device_status()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_keep_value_for_value(bs):
    rng = np.random.RandomState(bs)
    lens, rows, keep = [], [], []
    for r in [1, 1, 2, 16, 33, 64, 64, 7, 5, 0, 200]:
        rows.append(r)
        lens.append(r + int(rng.choice([0, 1, 15, 16, 64, 100])))
        pick = np.flatnonzero(rng.rand(r) < 0.5)[:64]
        keep.append(pick.tolist())
    keep[1], keep[5], keep[7], keep[8] = [0], list(range(64)), [6], []
    c = Cache(lens, 2, bs, seed=31, scale_exps=(-12, 3))
    dev, out, status = _keep(c, rows, keep)
    assert status == 0
    assert out == [n - r + len(k) for n, r, k in zip(lens, rows, keep)]
    oracle.kv8_keep(c.k, c.ks, c.tables, lens, rows, keep, bs)
    oracle.kv8_keep(c.v, c.vs, c.tables, lens, rows, keep, bs)
    assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)
    assert np.array_equal(dev[2].double().cpu().numpy(), c.ks)
    assert np.array_equal(dev[3].double().cpu().numpy(), c.vs)


@pytest.mark.parametrize("rows,keep", [
    ([4], [[2, 1]]), ([4], [[1, 1]]), ([4], [[0, 4]]), ([4], [[-1]]), ([70], [list(range(65))]),
    ([30], [[0]]),                       # more rows than keys
])
def test_keep_leaves_a_sequence_with_a_bad_list_alone(rows, keep):
    c = Cache([70 if rows[0] == 70 else 20], 1, 16, seed=32)
    dev, out, status = _keep(c, rows, keep)
    assert status == 6 and out == [-9]
    assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)


def test_keep_refuses_bad_tables_and_short_lists():
    c = Cache([20], 1, 16, seed=33)
    c.tables[0][1] = c.N
    dev, out, status = _keep(c, [8], [[5]])
    assert status == 6 and out == [-9] and np.array_equal(codes_of(dev[0]), c.k)
    c = Cache([20], 1, 16, seed=33)
    dev = c.device()                     # cu_keep says more entries than keep_idx has
    G.kv8_keep(*dev, i32([20]), i32([0, 8]), i32([0, 1]), i32([0, 3]))
    assert G.last_device_status() == 6 and np.array_equal(codes_of(dev[0]), c.k)
