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


def test_forked_compacted_cut_and_released():
    """A sequence of 9 pages and 5 tokens, of whose pages 1 to 5 three were given
    back: forked, compacted, shortened and released without a flag."""
    dev, nb = device(), 30
    row = [20, 7, -1, -1, 11, -1, 25, 3, 28, 14]
    tables = i32([row + [-1] * 2, [-1] * 12, [-1] * 12])
    lens, err = i32([149, -1, -1]), i32([0])
    free = [i for i in range(nb) if i not in row]
    stack, top, extra = i32(free + [-1] * (nb - len(free))), i32([len(free)]), i32([0] * nb)
    copies = torch.zeros(1, 2, dtype=torch.int64, device=dev)
    ops.xs_block_fork(i32([0]), i32([1]), tables, lens, stack, top, extra, copies, err_flag=err)
    last = free[-1]
    assert int(err) == 0 and copies.tolist() == [[14, last]] and lens.tolist() == [149, 149, -1]
    assert tables.tolist()[1] == row[:9] + [last, -1, -1]
    full = [i for i in row[:9] if i >= 0]
    assert extra.tolist() == [int(i in full) for i in range(nb)] and int(top) == len(free) - 1

    live = sorted(full + [14, last])
    L = len(live)
    holes, moved = [i for i in range(L) if i not in live], [i for i in live if i >= L]
    to = {i: i for i in live} | dict(zip(moved, holes)) | {-1: -1}
    remap, moves, count = i32([0] * nb), torch.zeros(nb // 2, 2, dtype=torch.int64, device=dev), i32([0])
    ops.xs_block_compact(tables, tables, lens, extra, extra, stack, top, remap, moves, count, err_flag=err)
    assert int(err) == 0 and int(top) == nb - L and int(count) == len(moved)
    row = [to[i] for i in row]
    assert tables.tolist() == [row + [-1] * 2, row[:9] + [to[last], -1, -1], [-1] * 12]
    assert extra.tolist() == [int(i in row[:9]) for i in range(nb)]

    # Shortened to 40 tokens: pages 3 (given back), 4, 5 (given back) and 6 to 9 are gone.
    ops.xs_block_truncate(i32([0]), i32([40]), tables, lens, stack, top, extra, err_flag=err)
    assert int(err) == 0 and lens.tolist() == [40, 149, -1] and tables.tolist()[0] == row[:3] + [-1] * 9
    assert extra.tolist() == [int(i in row[:2]) for i in range(nb)]
    assert int(top) == nb - L + 1 and stack.tolist()[nb - L] == row[9]
    before = int(top)
    ops.xs_block_release(i32([0, 1]), tables, lens, stack, top, extra, err_flag=err)
    assert int(err) == 0 and lens.tolist() == [-1] * 3 and extra.tolist() == [0] * nb
    gone = sorted([i for i in row[:9] if i >= 0] + [to[last]], reverse=True)
    assert int(top) == nb and stack.tolist()[before:nb] == gone


def test_other_ids_outside_the_pool_and_a_missing_last_page_are_told_of():
    dev = device()
    for bad in (-2, 8):
        tables, lens, err = i32([[3, bad, 1], [-1] * 3]), i32([40, -1]), i32([0])
        extra, stack, top = i32([0] * 8), i32([6] + [-1] * 7), i32([1])
        copies = torch.zeros(1, 2, dtype=torch.int64, device=dev)
        ops.xs_block_fork(i32([0]), i32([1]), tables, lens, stack, top, extra, copies, err_flag=err)
        assert int(err) == ops.FLAG_BAD_BLOCK
        for call in (lambda: ops.xs_block_truncate(i32([0]), i32([3]), tables, lens, stack, top, extra, err_flag=err),
                     lambda: ops.xs_block_release(i32([1]), tables, lens, stack, top, extra, err_flag=err)):
            err.zero_()
            call()
            assert int(err) == ops.FLAG_BAD_BLOCK
    tables, lens, err = i32([[3, 2, -1], [-1] * 3]), i32([40, -1]), i32([0])
    extra, stack, top = i32([0] * 8), i32([6] + [-1] * 7), i32([1])
    ops.xs_block_fork(i32([0]), i32([1]), tables, lens, stack, top, extra, copies, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK and copies.tolist() == [[-1, -1]]
