"""Shared pages: fork, release, compact and copy, against lists."""
import random

import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests import plain_ops as plain
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=device())


class Both:
    """A pool on the device and the same on lists."""

    def __init__(self, lens, width, nb, seed, capacity=None):
        rng = random.Random(seed)
        ids = list(range(nb))
        rng.shuffle(ids)
        tables, at = [], 0
        for n in lens:
            p = -(-n // 16) if n > 0 else 0
            tables.append(ids[at:at + p] + [-1] * (width - p))
            at += p
        stack = ids[at:] + [-1] * at
        self.top0 = nb - at
        cap = capacity or nb
        self.plain = plain.Pool(tables, lens, stack[:cap] + [-1] * max(0, cap - nb), self.top0, [0] * nb)
        self.tables, self.lens = i32(tables), i32(lens)
        self.stack, self.top = i32(self.plain.stack), i32([self.top0])
        self.extra, self.err = i32([0] * nb), i32([0])

    def check(self, what=""):
        p = self.plain
        assert self.lens.tolist() == p.lens, what
        assert self.tables.tolist() == p.tables, what
        assert int(self.top) == p.top and self.stack.tolist()[:p.top] == p.stack[:p.top], what
        assert self.extra.tolist() == p.extra, what
        assert int(self.err) == p.flags, what
        # every block has as many owners as it should
        owners = [0] * len(p.extra)
        for r, n in zip(p.tables, p.lens):
            for i in range(p.pages(n)):
                owners[r[i]] += 1
        for b in p.stack[:p.top]:
            assert owners[b] == 0, what
        assert [max(0, o - 1) for o in owners] == p.extra, what

    def fork(self, parents, children):
        n = len(parents)
        copies = torch.full((n, 2), 99, dtype=torch.int64, device=device())
        ops.xs_block_fork(i32(parents), i32(children), self.tables, self.lens, self.stack, self.top, self.extra,
                          copies, err_flag=self.err)
        assert copies.tolist() == [list(c) for c in self.plain.fork(parents, children)]
        return copies

    def release(self, ids):
        ops.xs_block_release(i32(ids), self.tables, self.lens, self.stack, self.top, self.extra, err_flag=self.err)
        self.plain.release(ids, self.stack.numel())


def test_fork_and_release():
    b = Both([33, 16, 0, 100, -1, -1, -1, -1, -1, -1, -1], 9, 40, seed=1)
    b.fork([0, 1, 2, 3, 0], [4, 5, 6, 7, 8])
    b.check("fork")
    b.fork([4, 8], [9, 10])                     # forks of forks
    b.check("fork of forks")
    b.release([0])                              # the first owner goes first
    b.check("parent")
    b.release([4, 5, 8, 1])
    b.check("some")
    b.release([9, 10, 7, 6, 2, 3])
    b.check("all")
    assert int(b.top) == 40
    assert b.stack.tolist()[:7] != sorted(b.stack.tolist()[:7])


def test_fork_skips_what_it_cannot_do():
    # ids out of range, a parent without a sequence, a child with one, a child
    # named twice (the first entry gets it), itself.
    b = Both([20, 5, -1, -1, -1, 7], 3, 12, seed=2)
    b.fork([-1, 0, 6, 0, 2, 0, 0, 1, 1, 5], [2, 6, 3, 1, 3, 3, 3, 3, 2, 5])
    assert b.plain.flags == ops.FLAG_BAD_SLOT
    b.check()


def test_fork_with_an_empty_stack():
    # 3 free blocks for 5 unfinished pages; entries in order, the others stay empty.
    b = Both([20, 32, -1, -1, -1, -1, -1, -1], 3, 7, seed=3)
    assert b.top0 == 3
    b.fork([0, 1, 0, 0, 0, 1], [2, 3, 4, 5, 6, 7])
    assert b.plain.flags == ops.FLAG_POOL_EMPTY and b.plain.lens == [20, 32, 20, 32, 20, 20, -1, 32]
    b.check()


def test_fork_of_a_parent_longer_than_its_table():
    b = Both([20, -1], 3, 8, seed=4)
    b.lens[0] = b.plain.lens[0] = 49
    b.fork([0], [1])
    assert b.plain.flags == ops.FLAG_BAD_LEN and int(b.lens[1]) == -1
    assert int(b.err) == ops.FLAG_BAD_LEN and int(b.top) == b.top0


def test_bad_blocks_are_flagged_and_not_counted():
    dev = device()
    tables = i32([[3, 99, 2, -1], [-1] * 4])
    lens, stack, top = i32([33, -1]), i32([7, 6]), i32([2])
    extra, err = i32([0] * 8), i32([0])
    copies = torch.zeros(1, 2, dtype=torch.int64, device=dev)
    ops.xs_block_fork(i32([0]), i32([1]), tables, lens, stack, top, extra, copies, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK and extra.tolist() == [0, 0, 0, 1, 0, 0, 0, 0]
    assert tables.tolist()[1] == [3, 99, 6, -1] and copies.tolist() == [[2, 6]]
    err.zero_()
    ops.xs_block_release(i32([1]), tables, lens, stack, top, extra, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK and extra.tolist() == [0] * 8
    assert int(top) == 2 and stack.tolist() == [7, 6]


def test_release_twice_empty_out_of_range_and_full():
    b = Both([33, 16, -1, 40], 4, 16, seed=5)
    b.release([1, 1, 2, -1, 4, 0])
    assert b.plain.flags == ops.FLAG_BAD_SLOT
    b.check()
    c = Both([33, 16], 4, 8, seed=6, capacity=6)        # 4 free, room for 2 of the 4 that come back
    c.release([0, 1])
    assert int(c.err) == ops.FLAG_POOL_EMPTY == c.plain.flags
    assert int(c.top) == 6 and c.stack.tolist() == c.plain.stack


@pytest.mark.parametrize("n,parents,width", [(1, 1, 1), (300, 7, 5), (2500, 40, 3)])
def test_large_forks(n, parents, width):
    rng = random.Random(n)
    lens = [rng.randrange(0, 16 * width + 1) for _ in range(parents)] + [-1] * n
    b = Both(lens, width, parents * width + n, seed=n)
    order = list(range(parents, parents + n))
    rng.shuffle(order)
    b.fork([rng.randrange(parents) for _ in order], order)
    b.check("fork")
    rng.shuffle(order)
    b.release(order[:n // 2])
    b.check("half")
    b.release(list(range(parents)) + order[n // 2:])
    b.check("all")


def test_same_result_every_time():
    # The order of the stack and of the copies does not depend on the run.
    seen = set()
    for _ in range(10):
        b = Both([45, 200, 31] + [-1] * 60, 16, 120, seed=7)
        b.fork([i % 3 for i in range(60)], list(range(3, 63)))
        b.release(list(range(0, 63, 2)))
        b.check()
        seen.add(tuple(b.stack.tolist()[:int(b.top)]))
    assert len(seen) == 1


def compacted(b, layers=2, H=2, D=64, inplace=False):
    dev = device()
    nb = b.extra.numel()
    k = torch.randint(0, 255, (layers, nb, H, 9 * D), dtype=torch.uint8, device=dev)
    v = torch.randint(0, 255, (layers, nb, H, 9 * D), dtype=torch.uint8, device=dev)
    k0, v0 = k.clone(), v.clone()
    t_out = b.tables if inplace else torch.full_like(b.tables, 55)
    e_out = b.extra if inplace else torch.full_like(b.extra, 55)
    remap, moves = i32([55] * nb), torch.full((nb // 2, 2), 55, dtype=torch.int64, device=dev)
    count = i32([55])
    before = [list(r) for r in b.plain.tables]
    want_remap, want_moves = b.plain.compact()
    ops.xs_block_compact(b.tables, t_out, b.lens, b.extra, e_out, b.stack, b.top, remap, moves, count,
                         err_flag=b.err)
    b.tables, b.extra = t_out, e_out
    assert remap.tolist() == want_remap and int(count) == len(want_moves)
    assert moves.tolist() == [list(m) for m in want_moves] + [[-1, -1]] * (nb // 2 - len(want_moves))
    b.check("compact")
    ops.xs_block_copy(k, v, moves, count=count, err_flag=b.err)
    for pool, was in ((k, k0), (v, v0)):
        for old, new, n in zip(before, b.plain.tables, b.plain.lens):
            p = b.plain.pages(n)
            assert torch.equal(pool[:, new[:p]], was[:, old[:p]])
    b.check("copied")


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("nb,seqs,live", [(1, 1, 1.0), (2, 1, 0.5), (33, 4, 0.4), (1000, 20, 0.6),
                                          (5000, 33, 0.93), (4096, 3, 0.02)])
def test_compact(nb, seqs, live, inplace):
    rng = random.Random(nb)
    per = max(1, int(nb * live) // seqs)
    lens = [rng.randrange(1, 16 * per + 1) for _ in range(seqs)] + [0, -1, -1, -1]
    width = per + 2
    b = Both(lens, width, nb, seed=nb)
    kids = [i for i, n in enumerate(lens) if n < 0][:2]
    if int(b.top) >= 2 and nb > 10:
        b.fork([0, 0], kids)
        b.release([0])
    compacted(b, inplace=inplace)
    compacted(b, inplace=inplace)               # nothing is left to move
    b.release(list(range(len(lens))))
    b.check("released")
    assert int(b.top) == nb


def test_compact_of_an_empty_pool_and_of_a_full_one():
    compacted(Both([-1, 0], 4, 9, seed=1))
    full = Both([16 * 5, 16 * 4], 6, 9, seed=2)
    compacted(full)
    assert int(full.top) == 0


def test_compact_flags():
    dev = device()
    tables, lens = i32([[3, 9, 1], [0, 5, 2]]), i32([48, 49])
    extra, err = i32([0] * 6), i32([0])
    out, e_out, stack, top = torch.zeros_like(tables), i32([7] * 6), i32([-5] * 6), i32([0])
    remap, moves, count = i32([0] * 6), torch.zeros(3, 2, dtype=torch.int64, device=dev), i32([0])
    ops.xs_block_compact(tables, out, lens, extra, e_out, stack, top, remap, moves, count, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK | ops.FLAG_BAD_LEN
    assert out.tolist() == [[3, 9, 1], [0, 4, 2]] and moves.tolist() == [[5, 4], [-1, -1], [-1, -1]]
    assert stack.tolist() == [5] + [-5] * 5 and int(top) == 1 and e_out.tolist() == [0] * 6


@pytest.mark.parametrize("shape,dtype", [((1, 5, 1, 16, 64), torch.bfloat16), ((3, 40, 8, 16, 128), torch.bfloat16),
                                         ((2, 9, 3, 16, 64), torch.float32), ((4, 11, 1, 9 * 64), torch.uint8)])
def test_copy(shape, dtype):
    dev = device()
    nb = shape[1]
    k, v = (torch.randint(0, 100, shape, device=dev).to(dtype) for _ in range(2))
    perm = torch.randperm(nb, generator=torch.Generator().manual_seed(nb)).tolist()
    pairs = [(perm[i], perm[i + 1]) for i in range(0, nb - 1, 2)]
    given = pairs + [(-1, 3), (2, -1), (nb, 0), (0, nb)]
    err = i32([0])
    wk, wv = k.clone(), v.clone()
    for s, d in pairs:
        for p in (wk, wv):
            p[:, d] = p[:, s]
    ops.xs_block_copy(k, v, torch.tensor(given, device=dev), err_flag=err)
    assert torch.equal(k, wk) and torch.equal(v, wv) and int(err) == ops.FLAG_BAD_BLOCK
    for count, done in ((0, 0), (1, 1), (-4, 0), (1000, len(pairs))):
        k2, v2 = (torch.randint(0, 100, shape, device=dev).to(dtype) for _ in range(2))
        wk, wv = k2.clone(), v2.clone()
        for s, d in pairs[:done]:
            for p in (wk, wv):
                p[:, d] = p[:, s]
        ops.xs_block_copy(k2, v2, torch.tensor(pairs, device=dev), count=i32([count]))
        assert torch.equal(k2, wk) and torch.equal(v2, wv)


def test_copy_far_layers():
    # Layers whose offsets pass 2^32 bytes.
    dev = device()
    k = torch.empty(3, 1000, 1 << 17, 16, dtype=torch.uint8, device=dev)     # 2.1 GB a layer
    k[:, 998], k[:, 7] = 5, 1
    ops.xs_block_copy(k, k.clone(), torch.tensor([[998, 7]], device=dev))
    assert bool((k[:, 7] == 5).all()) and bool((k[:, 998] == 5).all())


def test_with_the_allocator_and_a_graph():
    """A captured step: allocate, append, with forks in between; the allocator
    and the shared counts work on one state."""
    dev = device()
    nb, B, H, D = 64, 6, 2, 64
    k, v = (torch.zeros(1, nb, H, 16, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
    tables, lens = torch.full((B, 8), -1, dtype=torch.int32, device=dev), i32([0, 0, -1, -1, -1, -1])
    stack, top, extra, err = i32(list(range(nb - 1, -1, -1))), i32([nb]), i32([0] * nb), i32([0])
    rows = torch.zeros(B, H, D, dtype=torch.bfloat16, device=dev)
    def one():
        ops.xs_block_alloc_decode(tables, lens, stack, top, err_flag=err)
        ops.xs_kv_append_paged(rows, rows, k[0], v[0], tables, lens, err_flag=err)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            one()
    torch.cuda.current_stream().wait_stream(s)
    said = {b: [] for b in range(B)}
    value = 0
    copies = torch.empty(2, 2, dtype=torch.int64, device=dev)

    def steps(count):
        nonlocal value
        for _ in range(count):
            value += 1
            rows.copy_((value + 200 * torch.arange(B, device=dev))[:, None, None].expand(B, H, D) % 251)
            graph.replay()
            for b in range(B):
                if int(lens[b]) > 0:
                    said[b].append((value + 200 * b) % 251)

    steps(21)
    ops.xs_block_fork(i32([0, 0]), i32([2, 4]), tables, lens, stack, top, extra, copies, err_flag=err)
    ops.xs_block_copy(k, v, copies, err_flag=err)
    said[2], said[4] = list(said[0]), list(said[0])
    steps(30)
    ops.xs_block_release(i32([0]), tables, lens, stack, top, extra, err_flag=err)
    ops.xs_block_fork(i32([4]), i32([0]), tables, lens, stack, top, extra, copies[:1], err_flag=err)
    ops.xs_block_copy(k, v, copies[:1], err_flag=err)
    said[0] = list(said[4])
    steps(14)
    remap, moves, count = i32([0] * nb), torch.empty(nb // 2, 2, dtype=torch.int64, device=dev), i32([0])
    ops.xs_block_compact(tables, tables, lens, extra, extra, stack, top, remap, moves, count, err_flag=err)
    ops.xs_block_copy(k, v, moves, count=count, err_flag=err)
    steps(9)
    assert int(err) == 0
    for b in (0, 1, 2, 4):
        n = int(lens[b])
        assert n == len(said[b]) > 0
        got = k[0, tables[b, :-(-n // 16)].long()].transpose(1, 2).flatten(0, 1)[:n, 0, 0]
        assert got.tolist() == said[b]
