"""The debug library's bounds checks in the norm + rotation, 4-bit cache and
shared-page kernels: none fails in calls of many shapes, and one that must
fail is counted, flagged, and its access left out."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import Kv4DecodeStep
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
FLAG_BOUNDS = 64


@pytest.fixture()
def debug():
    device()
    xsbuild.build(debug_bounds=True)
    lib = ops.load_debug()
    prev = ops.use_library(lib)
    try:
        ops.xs_debug_bounds_failures(reset=True, lib=lib)
        yield lib
    finally:
        ops.use_library(prev)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=device())


def test_a_stack_top_beyond_the_pool_is_counted(debug):
    # Four blocks in the pool and a top of six, in a stack that has the room:
    # no read is out of the buffer's memory, but the sixth entry is not one.
    tables, lens = i32([[0, 1], [-1, -1], [-1, -1]]), i32([20, -1, -1])
    stack, top, extra, err = i32([3, 2, 3, 2, 3, 2]), i32([6]), i32([0] * 4), i32([0])
    copies = torch.zeros(1, 2, dtype=torch.int64, device=device())
    ops.xs_block_fork(i32([0]), i32([1]), tables, lens, stack, top, extra, copies, err_flag=err)
    assert int(err) == FLAG_BOUNDS | ops.FLAG_BAD_BLOCK
    assert ops.xs_debug_bounds_failures(reset=True, lib=debug) == 1
    assert copies.tolist() == [[-1, -1]] and tables.tolist()[1] == [0, -1]


@pytest.mark.parametrize("B,Hq,Hkv,D,rot", [(1, 8, 8, 64, 32), (9, 64, 8, 128, 128), (70, 8, 2, 128, 48)])
def test_a_step_and_a_pool_without_failures(debug, B, Hq, Hkv, D, rot):
    dev, width = device(), 40
    nb = B * width + B
    g = torch.Generator(device=dev).manual_seed(B)
    kc, vc = ops.kv4_pools(nb, Hkv, D, dev, layers=1)
    tables = torch.full((2 * B, width), -1, dtype=torch.int32, device=dev)
    lens = torch.full((2 * B,), -1, dtype=torch.int32, device=dev)
    stack, top = torch.arange(nb - 1, -1, -1, dtype=torch.int32, device=dev), i32([nb])
    extra, err = i32([0] * nb), i32([0])
    tab = ops.rope_table(16 * width, rot, 1e4, dev)
    step = Kv4DecodeStep(2 * B, Hq, Hkv, D, dev, window=200)
    lens[:B] = 0
    out = torch.empty(2 * B, Hq, D, dtype=BF, device=dev)
    copies = torch.empty(B, 2, dtype=torch.int64, device=dev)

    def steps(n):
        for _ in range(n):
            x = torch.randn(2 * B, Hq + 2 * Hkv, D, generator=g, device=dev).to(BF)
            ops.xs_block_alloc_decode(tables, lens, stack, top, err_flag=err)
            step.run(out, *x.split([Hq, Hkv, Hkv], 1), None, None, tab, kc[0], vc[0], tables, lens, 0.1)

    steps(35)
    ops.xs_block_fork(torch.arange(B, dtype=torch.int32, device=dev),
                      torch.arange(B, 2 * B, dtype=torch.int32, device=dev), tables, lens, stack, top, extra,
                      copies, err_flag=err)
    ops.xs_block_copy(kc, vc, copies, err_flag=err)
    steps(20)
    ops.xs_block_release(torch.arange(0, 2 * B, 2, dtype=torch.int32, device=dev), tables, lens, stack, top, extra,
                         err_flag=err)
    remap, moves, count = i32([0] * nb), torch.empty(nb // 2, 2, dtype=torch.int64, device=dev), i32([0])
    ops.xs_block_compact(tables, tables, lens, extra, extra, stack, top, remap, moves, count, err_flag=err)
    ops.xs_block_copy(kc, vc, moves, count=count, err_flag=err)
    steps(20)
    ko, vo = (torch.empty(B, Hkv, 16, D, dtype=BF, device=dev) for _ in range(2))
    ops.xs_kv4_unpack(ko, vo, kc[0], vc[0], torch.arange(B, dtype=torch.int32, device=dev), err_flag=err)
    assert int(err) == 0 and step.error_flags() == 0
    assert ops.xs_debug_bounds_failures(reset=True, lib=debug) == 0
