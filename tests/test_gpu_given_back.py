"""Tables some of whose pages were given back (-1), as under a window."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests.gpu_helpers import device
from tests.test_gpu_share import i32

pytestmark = pytest.mark.gpu


def test_free_pushes_no_negative_ids():
    tables, lens = i32([[3, -1, -1, 5], [-1, 6, -7, 1], [2, -1, -1, -1]]), i32([60, 49, 3])
    stack, top, err = i32([0] + [9] * 9), i32([1]), i32([0])
    ops.xs_block_free(i32([0]), tables, lens, stack, top, err_flag=err)
    assert int(top) == 3 and sorted(stack.tolist()[:3]) == [0, 3, 5] and stack.tolist()[3:] == [9] * 7
    assert int(err) == 0 and tables.tolist()[0] == [-1] * 4 and lens.tolist() == [-1, 49, 3]
    ops.xs_block_free(i32([1, 2]), tables, lens, stack, top, err_flag=err)
    assert int(top) == 6 and sorted(stack.tolist()[:6]) == [0, 1, 2, 3, 5, 6]
    assert int(err) == ops.FLAG_BAD_BLOCK and lens.tolist() == [-1] * 3
    # What the allocator hands out next is a block.
    lens.zero_()
    ops.xs_block_alloc_decode(tables, lens, stack, top, err_flag=err)
    assert sorted(t[0] for t in tables.tolist()) == sorted(set(range(7)) - {4} - set(stack.tolist()[:3]))
