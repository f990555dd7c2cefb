"""Appends with several runs of rows in one block: rows skipped in the middle of a sequence and
sequences whose tokens alternate, code for code against the oracle, which takes the runs in order."""
import numpy as np
import pytest
import torch

import gqa_head_gated_gb300 as G
import oracle
from tests.kv8_cases import DEV, Cache, codes_of, i32
from tests.test_gpu_kv8_cache import _append, _new, _slots

pytestmark = pytest.mark.gpu


def _spread(n, Hkv, seed, dtype, big=()):
    """Rows whose largest values differ by powers of two; rows `big` by far more than those before."""
    x, y = _new(n, Hkv, seed, dtype, spread=3.0)
    for i in big:
        x[i] *= 64
        y[i] *= 32
    return x, y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("held", [0, 5])
def test_a_skipped_row_inside_a_block(held, bs, dtype):
    """Slots [s, -1, s + 1] behind held rows and in an empty block, growing and not."""
    c = Cache([held] * 8, 3, bs, seed=131, room=16)
    slots = []
    for b in range(8):
        a = _slots(c, b, held, 4)
        slots += [a[0], -1, a[1], -1, -1, a[2], a[3]] if b % 2 else [a[0], a[1], -1, a[3]]
    x, y = _spread(len(slots), 3, 132, dtype, big=[2, 11, 20, 31])
    assert _append(c, x, y, slots) == 0


@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("at", [61, 62, 63, 64, 65, 127, 128])
def test_runs_of_a_block_on_both_sides_of_a_window(at, bs):
    """The rows of one block before and behind token `at`, with a skipped row between them."""
    c = Cache([3, 5], 2, bs, seed=133, room=at + 16)
    lead = _slots(c, 1, 5, at - 2)              # other rows, so that the block's start at token at - 2
    a = _slots(c, 0, 3, 8)
    slots = lead + [a[0], a[1], -1, a[2], -1, -1, a[5], a[6]]
    x, y = _spread(len(slots), 2, 134, torch.bfloat16, big=[at + 1, at + 5])
    assert _append(c, x, y, slots) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("bs,B,n", [(16, 2, 200), (64, 3, 150), (128, 7, 60), (32, 40, 9)])
def test_sequences_whose_tokens_alternate(B, n, bs, dtype):
    held = [(7 * b) % 23 for b in range(B)]
    c = Cache(held, 2, bs, seed=135, room=n)
    per = [_slots(c, b, held[b], n) for b in range(B)]
    slots = [per[b][i] for i in range(n) for b in range(B)]
    x, y = _spread(len(slots), 2, 136, dtype, big=range(37, len(slots), 53))
    assert _append(c, x, y, slots) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B", [2, 5, 11, 20, 30])
def test_a_small_step_of_many_sequences(B, dtype):
    """A row each of up to 30 sequences, and behind them another of one or two."""
    c = Cache([5 + b for b in range(B)], 2, 64, seed=145, room=8)
    slots = [_slots(c, b, 5 + b, 1)[0] for b in range(B)]
    for again in ([0], [B - 2], [B // 2, 0]):
        more = slots + [_slots(c, b, 6 + b, 1)[0] for b in again]
        x, y = _spread(len(more), 2, 146, dtype, big=[len(more) - 1])
        assert _append(c, x, y, more) == 0


def test_every_third_row_skipped_and_far_apart():
    """A sequence with a third of its rows left out, and a block whose second run lies thousands of
    tokens behind its first."""
    c = Cache([0, 9], 2, 64, seed=137, room=6200)
    a, far = _slots(c, 0, 0, 6000), _slots(c, 1, 9, 30)
    slots = far[:3] + [s if i % 3 else -1 for i, s in enumerate(a)] + far[3:11] + [-1] + far[11:30]
    x, y = _spread(len(slots), 2, 138, torch.bfloat16, big=[1500, 6004, 6013])
    assert _append(c, x, y, slots) == 0


def test_nan_and_infinities_in_a_later_run():
    c = Cache([4], 2, 16, seed=139, room=12)
    a = _slots(c, 0, 4, 12)
    x, y = _spread(10, 2, 140, torch.bfloat16, big=[4])
    x[2, 0, 5], x[2, 1, 7], y[4, 0, 0], y[6] = float("nan"), float("inf"), -float("inf"), 0.0
    assert _append(c, x, y, [a[0], -1, a[1], a[2], -1, a[4], -1, a[9], a[10], a[11]]) == 0


@pytest.mark.parametrize("between", [1, 70, 300])
def test_rows_that_come_again_are_skipped_and_recorded(between):
    """The same row twice, a row before one that was written, and a run behind a block's last row: the
    cache is as if they were not there."""
    c = Cache([3, 3, 3, 0], 2, 16, seed=141, room=400)
    a, b, d = (_slots(c, i, 3, 13) for i in range(3))
    rest = _slots(c, 3, 0, between)             # tokens between the runs
    bad = [a[4], a[5]], [b[2]], [d[1], d[2]]    # again; behind row 3 + 4; behind the last row
    slots = a[4:6] + [-1] + b[4:5] + [-1] + d + rest
    good = list(slots)
    for r in bad:
        slots += [-1] + r
        good += [-1] * (1 + len(r))
    slots += [-1] + a[6:8] + [-1] + b[5:6]      # in order again
    good += [-1] + a[6:8] + [-1] + b[5:6]
    x, y = _spread(len(slots), 2, 142, torch.bfloat16, big=[1, len(slots) - 1])
    dev = c.device()
    G.kv8_append(x.to(DEV), y.to(DEV), i32(slots), *dev[:4])
    assert G.last_device_status() == 6
    oracle.kv8_append(c.k, c.ks, x.double().numpy(), good, 16)
    oracle.kv8_append(c.v, c.vs, y.double().numpy(), good, 16)
    assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)
    for t, s in zip(dev[2:4], (c.ks, c.vs)):
        assert np.array_equal(t.double().cpu().numpy(), s)


def test_many_runs_captured_and_replayed():
    c = Cache([2] * 20, 2, 32, seed=143, room=30)
    slots = [s for i in range(10) for b in range(20) for s in (_slots(c, b, 2 + 2 * i, 1) + [-1])]
    x, y = _spread(len(slots), 2, 144, torch.bfloat16, big=[150, 330])
    dev = c.device()
    start = [t.view(torch.uint8).clone() for t in dev[:4]]
    xd, yd, sd = x.to(DEV), y.to(DEV), i32(slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.kv8_append(xd, yd, sd, *dev[:4])
    oracle.kv8_append(c.k, c.ks, x.double().numpy(), slots, 32)
    oracle.kv8_append(c.v, c.vs, y.double().numpy(), slots, 32)
    for _ in range(3):
        for t, s in zip(dev[:4], start):
            t.view(torch.uint8).copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(codes_of(dev[0]), c.k) and np.array_equal(codes_of(dev[1]), c.v)
    assert G.last_device_status() == 0
