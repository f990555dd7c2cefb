"""Forks from tables and stacks that name no block of the pool: recorded, and no copy of such a one listed."""
import pytest

import gqa_head_gated_gb300 as G
from tests.kv8_cases import i32

pytestmark = pytest.mark.gpu


def _state():
    """8 blocks of 16 keys: sequence 0 holds 40 keys in 3, 1, 6; 1 and 2 nothing."""
    return dict(lens=i32([40, 0, 0]), tables=i32([[3, 1, 6, -1]] + [[-1] * 4] * 2), n=i32([3, 0, 0]),
                free=i32([0, 2, 4, 5, 7, -1, -1, -1]), fc=i32([5]), shares=i32([0] * 8))


def _fork(d, src, dst, lens):
    return G.block_fork(i32(src), i32(dst), i32(lens), d["lens"], d["tables"], d["n"], d["free"], d["fc"], d["shares"], 16)


@pytest.mark.parametrize("entry", [-1, 8, 77, -2 ** 31, 2 ** 31 - 1])
def test_a_parent_whose_last_entry_is_no_block(entry):
    d = _state()
    d["tables"][0, 2] = entry
    copies = _fork(d, [0, 0], [1, 2], [35, 20])
    assert G.last_device_status() == 6
    assert copies.tolist() == [[-1, -1, 0], [1, 5, 4]]
    assert d["tables"].tolist() == [[3, 1, entry, -1], [3, 1, 7, -1], [3, 5, -1, -1]]
    assert d["shares"].tolist() == [0, 1, 0, 2, 0, 0, 0, 0] and d["fc"].item() == 3


@pytest.mark.parametrize("entry", [-1, 8, 2 ** 31 - 1])
def test_a_stack_whose_top_is_no_block(entry):
    d = _state()
    d["free"][4] = entry
    copies = _fork(d, [0, 0], [1, 2], [35, 20])
    assert G.last_device_status() == 6
    assert copies.tolist() == [[-1, -1, 0], [1, 5, 4]]
    assert d["tables"].tolist() == [[3, 1, 6, -1], [3, 1, -1, -1], [3, 5, -1, -1]]
    assert d["n"].tolist() == [3, 3, 2] and d["fc"].item() == 3
