"""Eviction by accumulated weight, truncation, and whole bounded decode steps."""
import random

import numpy as np
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import BoundedDecodeStep
from tests import plain_bounded as plain
from tests.gpu_helpers import device
from tests.test_gpu_share import Both, i32

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class State:
    def __init__(self, lens, layers, Hkv, D, dtype, seed, width=None, draw="spread"):
        self.g = g = torch.Generator().manual_seed(seed)
        pages = [-(-max(n, 0) // 16) for n in lens]
        width = width or max(pages + [1])
        nb = sum(pages) + 2
        perm = torch.randperm(nb, generator=g).tolist()
        self.tables = torch.full((len(lens), width), -1, dtype=torch.int32)
        for b, p in enumerate(pages):
            for c in range(p):
                self.tables[b, c] = perm.pop()
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.k, self.v = (torch.randn(layers, nb, Hkv, 16, D, generator=g).to(dtype) for _ in range(2))
        x = torch.randn(layers, len(lens), Hkv, width * 16, generator=g)
        if draw == "spread":
            x = (3 * x).exp()
        elif draw == "ties":
            x = x.round() * 0.5
        elif draw == "equal":
            x.fill_(0.25)
        elif draw == "odd":
            odd = torch.tensor([float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-45, -1e-45, -3.0, 3e38])
            x = torch.where(torch.rand(x.shape, generator=g) < 0.6, odd[torch.randint(0, 9, x.shape, generator=g)], x)
        self.scores = x
        self.err = i32([0])

    def run(self, ids, first, recent, budget, limit, extra=None):
        dev = device()
        bits = np.int16 if self.k.element_size() == 2 else np.int32
        as_bits = lambda t: t.cpu().contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32).numpy()  # noqa: E731
        want = plain.Evicted(ids, as_bits(self.k), as_bits(self.v), self.scores.numpy(), self.tables.tolist(),
                             self.lens.tolist(), first, recent, budget, limit, extra)
        k, v, s = self.k.to(dev), self.v.to(dev), self.scores.to(dev)
        L, B, Hkv, _ = s.shape
        kept = torch.full((L, len(ids), Hkv, budget), 77, dtype=torch.int32, device=dev)
        new = i32([77] * len(ids))
        ops.xs_kv_evict(i32(ids), k, v, s, self.tables.to(dev), self.lens.to(dev), kept, new, first, recent, limit,
                        extra_refs=None if extra is None else i32(extra), err_flag=self.err)
        assert new.tolist() == want.new_lens.tolist()
        assert np.array_equal(kept.cpu().numpy(), want.kept)
        assert np.array_equal(s.cpu().numpy().view(np.int32), want.scores.view(np.int32))
        assert np.array_equal(as_bits(k), want.k) and np.array_equal(as_bits(v), want.v)
        assert int(self.err) == want.flags
        assert bits is not None
        return want


@pytest.mark.parametrize("draw", ["spread", "ties", "equal", "odd"])
@pytest.mark.parametrize("first,recent,budget,limit", [(4, 8, 30, 30), (0, 0, 1, 1), (0, 0, 47, 60), (5, 20, 25, 40),
                                                       (33, 0, 33, 50), (0, 16, 16, 16), (17, 3, 64, 64), (1, 1, 120, 130)])
def test_evict(draw, first, recent, budget, limit):
    lens = [0, 31, 200, -1, 131, 64, 1, 65, 129, 130]
    s = State(lens, 2, 2, 64, BF, budget, draw=draw)
    s.run([4, 0, 9, 2, 3, 8, 1, 5], first, recent, budget, limit)


@pytest.mark.parametrize("layers,Hkv,D,dtype", [(1, 1, 64, BF), (3, 2, 128, F32), (1, 8, 128, BF), (2, 3, 64, F32)])
def test_types_and_heads(layers, Hkv, D, dtype):
    s = State([700, 90, 333, 1, 400], layers, Hkv, D, dtype, D + layers, width=60)
    s.run([0, 1, 2, 3, 4], 4, 50, 128, 200)


@pytest.mark.parametrize("n,width,budget", [(5000, 313, 300), (40000, None, 2000), (60000, None, 777), (4096, 257, 4095)])
def test_long(n, width, budget):
    # Scores held by 1,024 threads, and more than shared memory holds.
    s = State([n, 100], 1, 1, 64, BF, n, width=width, draw="ties" if n == 40000 else "spread")
    s.run([1, 0], 4, 100, budget, budget)


@pytest.mark.parametrize("n,budget,recent,draw", [(70000, 3001, 1500, "spread"), (70000, 9000, 40, "ties"), (66000, 65999, 7, "equal"),
                                                  (170001, 2500, 900, "odd")])
def test_very_long(n, budget, recent, draw):
    # Each warp has more positions than it looks at at a time; more scores than shared memory holds.
    s = State([n, 50], 1, 1, 64, BF, budget, draw=draw)
    s.run([1, 0], 4, recent, budget, budget)


def test_entries_that_are_not_cut():
    s = State([100, 100, 100, 100, 100, 300], 1, 2, 64, BF, 3)
    extra = [0] * s.k.shape[1]
    extra[int(s.tables[1, 2])] = 1          # a page that would be written is shared
    extra[int(s.tables[2, 5])] = 1          # one behind the budget is
    extra[int(s.tables[3, 0])] = 2          # one of whole first tokens is
    s.tables[4, 6] = -1                     # a page that would be read has no block
    w = s.run([0, 1, 2, 3, 4, 6, 0, -1, 5], 16, 10, 50, 50, extra)
    assert w.new_lens.tolist() == [50, -1, 50, 50, -1, -1, -1, -1, 50]
    assert w.flags == ops.FLAG_SHARED | ops.FLAG_BAD_BLOCK | ops.FLAG_BAD_SLOT
    s = State([100, 100], 1, 2, 64, BF, 4)
    extra = [0] * s.k.shape[1]
    extra[int(s.tables[0, 1])] = 1          # shared, but nothing is written: the first tokens alone are kept
    assert s.run([0, 1], 20, 0, 20, 20, extra).new_lens.tolist() == [20, 20]
    s = State([100, 90], 1, 2, 64, BF, 3, width=7)
    s.lens[0] = 200                         # beyond its table: the table's 112
    for c in range(7):
        s.tables[0, c] = c
    assert s.run([0, 1], 0, 0, 20, 95).flags == ops.FLAG_BAD_LEN


def test_evict_captured_behind_other_work():
    s = State([90, 200], 1, 2, 64, BF, 9)
    dev = device()
    k, v, sc = s.k.to(dev), s.v.to(dev), s.scores.to(dev)
    tables, lens, ids = s.tables.to(dev), s.lens.to(dev), i32([1, 0])
    kept, new = torch.empty(1, 2, 2, 40, dtype=torch.int32, device=dev), i32([0, 0])
    call = lambda: ops.xs_kv_evict(ids, k, v, sc, tables, lens, kept, new, 2, 10, 60)  # noqa: E731
    call()
    want = kept.clone(), k.clone(), sc.clone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(2):
        k.copy_(s.k), v.copy_(s.v), sc.copy_(s.scores)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want[0]) and torch.equal(k, want[1]) and torch.equal(sc, want[2])
    assert new.tolist() == [40, 40]


# ---------------------------------------------------------------- truncation

class Cut(Both):
    def truncate(self, ids, new):
        ops.xs_block_truncate(i32(ids), i32(new), self.tables, self.lens, self.stack, self.top, self.extra,
                              err_flag=self.err)
        plain.truncate(self.plain, ids, new)


@pytest.mark.parametrize("nb,width", [(60, 12), (5000, 40), (50000, 12)])
def test_truncate(nb, width):
    s = Cut([100, 33, 0, 16, -1, 150, -1, 20], width, nb, nb)
    s.truncate([5], [149])                  # within the last page
    s.check("a page's end")
    s.truncate([0, 1, 3], [64, 1, 16])
    s.check("three")
    s.truncate([0, 1, 2, 3, 4, 5, 7], [0, 5, 3, -1, 0, 20, 0])
    s.check("to zero, longer, empty, left alone")
    s.truncate([5, 9, 5, -1, 5], [17, 0, 3, 0, 1])
    s.check("ids that are not, or twice")
    assert int(s.err) == ops.FLAG_BAD_SLOT and s.lens.tolist()[5] == 17


@pytest.mark.parametrize("nb,n,width", [(300000, 40, 700), (41000, 64, 640), (263000, 3, 11)])
@pytest.mark.parametrize("release", [False, True], ids=["truncate", "release"])
def test_given_back_from_large_pools(nb, n, width, release):
    # More block ids than each warp looks at at a time, some with a second owner.
    g = torch.Generator().manual_seed(nb + n)
    tables = torch.randperm(nb, generator=g)[:n * width].view(n, width).to(torch.int32)
    lens = torch.full((n,), width * 16, dtype=torch.int32)
    new = torch.randint(0, width * 16, (n,), generator=g).to(torch.int32)
    extra = (torch.rand(nb, generator=g) < 0.2).to(torch.int32)
    pages = torch.zeros_like(new) if release else -(-new // 16)
    gone = torch.cat([tables[b, int(pages[b]):] for b in range(n)]).long()
    want_extra, want_tables = extra.clone(), tables.clone()
    want_extra[gone] -= 1
    free = sorted((i for i in gone.tolist() if want_extra[i] < 0), reverse=True)
    want_extra.clamp_(min=0)
    for b in range(n):
        want_tables[b, int(pages[b]):] = -1
    stack, top, err = torch.full((nb,), 7, dtype=torch.int32, device=device()), i32([5]), i32([0])
    t, x, c, ids = tables.to(device()), extra.to(device()), lens.to(device()), torch.arange(n, dtype=torch.int32, device=device())
    if release:
        ops.xs_block_release(ids, t, c, stack, top, x, err_flag=err)
    else:
        ops.xs_block_truncate(ids, new.to(device()), t, c, stack, top, x, err_flag=err)
    assert int(top) == 5 + len(free) and int(err) == 0
    assert stack[:5 + len(free)].tolist() == [7] * 5 + free and bool((stack[5 + len(free):] == 7).all())
    assert torch.equal(x.cpu(), want_extra) and torch.equal(t.cpu(), want_tables)
    assert torch.equal(c.cpu(), torch.full_like(new, -1) if release else new)


def test_truncate_shared_pages():
    s = Cut([100, 70, -1, -1, -1], 8, 40, 3)
    s.fork([0, 0, 1], [2, 3, 4])
    s.check("forked")
    s.truncate([0, 2], [20, 40])
    s.check("two of three owners")
    s.truncate([3, 4, 1], [0, 16, 65])
    s.check("the last owners")


def test_truncate_into_a_full_stack_and_bad_blocks():
    s = Cut([64, 64], 4, 12, 5, capacity=6)
    s.truncate([0], [10])
    assert int(s.err) == ops.FLAG_POOL_EMPTY and int(s.top) == 6 and s.lens.tolist() == [10, 64]
    s = Cut([64, 64], 4, 12, 5)
    s.tables[1, 3] = 99
    s.plain.tables[1][3] = 99
    s.truncate([1], [10])
    assert int(s.err) == ops.FLAG_BAD_BLOCK and s.tables.tolist() == s.plain.tables
    assert s.stack.tolist()[:int(s.top)] == s.plain.stack[:s.plain.top]


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("dtype,Hq,Hkv,D", [(BF, 8, 2, 128), (F32, 4, 4, 64)])
def test_bounded_steps(dtype, Hq, Hkv, D):
    """Two layers of a decode loop whose sequences are bounded: each attention
    against 64 bits on the rows that were kept (their texts' own), each choice
    against the scores it was made from, each length and page accounted for."""
    dev, layers, B, budget, limit, first, recent = device(), 2, 3, 40, 48, 2, 10
    rng, width, nb = random.Random(1), 6, 20
    g = torch.Generator(device=dev).manual_seed(4)
    step = BoundedDecodeStep(B, Hq, Hkv, D, width, layers, dtype, dev, budget, limit, first, recent)
    k, v = (torch.zeros(layers, nb, Hkv, 16, D, dtype=dtype, device=dev) for _ in range(2))
    tables, lens = torch.full((B, width), -1, dtype=torch.int32, device=dev), i32([0, 0, -1])
    stack, top, extra = i32(list(range(nb))), i32([nb]), i32([0] * nb)
    table = ops.rope_table(400, D, 1e4, dev)
    w = torch.ones(D, dtype=dtype, device=dev) + 0.1 * torch.randn(D, generator=g, device=dev).to(dtype)
    texts = [[[[] for _ in range(Hkv)] for _ in range(B)] for _ in range(layers)]    # positions held, by layer, slot, head
    all_k, all_v = ([[] for _ in range(layers)] for _ in range(2))
    pos = [0, 0, 0]
    out = torch.empty(B, Hq, D, dtype=dtype, device=dev)
    evictions = 0
    for t in range(75):
        if t == 9:
            lens[2] = 0
            step.start([2])
        ops.xs_block_alloc_decode(tables, lens, stack, top)
        live = [b for b in range(B) if int(lens[b]) > 0]
        positions = i32([pos[b] if b in live else -1 for b in range(B)])
        for l in range(layers):
            x = torch.randn(B, Hq + 2 * Hkv, D, generator=g, device=dev).to(dtype)
            before = step.scores[l].clone()
            step.run(l, out, *x.split([Hq, Hkv, Hkv], 1), w, w, table, positions, k[l], v[l], tables, lens, D ** -0.5)
            rk = torch.empty(B, Hkv, D, dtype=dtype, device=dev)
            rq = torch.empty(B, Hq, D, dtype=dtype, device=dev)
            ops.xs_qk_norm_rope(rq, rk, x[:, :Hq], x[:, Hq:Hq + Hkv], w, w, 1e-6, table, positions)
            all_k[l].append(rk.cpu()), all_v[l].append(x[:, Hq + Hkv:].cpu())
            for b in live:
                n = int(lens[b])
                for h in range(Hkv):
                    texts[l][b][h].append(t)
                    held = texts[l][b][h]
                    assert len(held) == n
                    kk = torch.stack([all_k[l][i][b, h] for i in held])[:, None].double()
                    vv = torch.stack([all_v[l][i][b, h] for i in held])[:, None].double()
                    heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
                    o, p, mag, slack = plain.attend(rq[b, heads].cpu(), kk, vv, D ** -0.5)
                    bound = plain.out_bound(o, mag, slack, dtype, 15 if dtype == BF else 20)
                    assert bool(((out[b, heads].cpu().double() - o).abs() <= bound).all()), (t, l, b, h)
                    old = before[b, h, :n].cpu().double()
                    old[n - 1] = 0
                    assert torch.allclose(step.scores[l, b, h, :n].cpu().double(), old + p.sum(0), atol=1e-5)
        scores, n0 = step.scores.cpu(), lens.tolist()
        step.bound(k, v, tables, lens, stack, top, extra)
        for b in live:
            pos[b] += 1
            if n0[b] <= limit:
                assert int(lens[b]) == n0[b]
                continue
            evictions += 1
            assert int(lens[b]) == budget
            for l in range(layers):
                for h in range(Hkv):
                    at = plain.keep(scores[l, b, h].tolist(), n0[b], first, recent, budget)
                    assert step.kept[l, b, h].tolist() == at
                    texts[l][b][h] = [texts[l][b][h][i] for i in at]
        used = sum(-(-max(int(x), 0) // 16) for x in lens)
        assert int(top) == nb - used
        assert step.scored.tolist() == lens.tolist()
    assert evictions >= 6 and step.error_flags() == 0
    assert rng is not None


def test_bounded_steps_captured():
    """A step of two layers with its eviction as one graph, replayed over lengths
    that reach the limit again and again: the same as the calls one by one."""
    dev, layers, B, Hq, Hkv, D, width, nb = device(), 2, 3, 8, 2, 64, 6, 20
    g = torch.Generator(device=dev).manual_seed(6)
    x = torch.randn(60, layers, B, Hq + 2 * Hkv, D, generator=g, device=dev).to(BF)
    table = ops.rope_table(100, D, 1e4, dev)
    w = torch.ones(D, dtype=BF, device=dev)

    class Loop:
        def __init__(self):
            self.step = BoundedDecodeStep(B, Hq, Hkv, D, width, layers, BF, dev, 40, 44, 2, 10)
            self.k, self.v = (torch.zeros(layers, nb, Hkv, 16, D, dtype=BF, device=dev) for _ in range(2))
            self.tables, self.lens = torch.full((B, width), -1, dtype=torch.int32, device=dev), i32([0, 0, -1])
            self.stack, self.top, self.extra = i32(list(range(nb))), i32([nb]), i32([0] * nb)
            self.pos, self.x = i32([0, 0, -1]), torch.empty_like(x[0])
            self.out = torch.zeros(layers, B, Hq, D, dtype=BF, device=dev)

        def run(self):
            ops.xs_block_alloc_decode(self.tables, self.lens, self.stack, self.top)
            for l in range(layers):
                self.step.run(l, self.out[l], *self.x[l].split([Hq, Hkv, Hkv], 1), w, w, table, self.pos, self.k[l],
                              self.v[l], self.tables, self.lens, D ** -0.5)
            self.step.bound(self.k, self.v, self.tables, self.lens, self.stack, self.top, self.extra)

    eager, captured = Loop(), Loop()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured.run()
    shortened = 0
    for t in range(60):
        for loop in (eager, captured):
            loop.x.copy_(x[t])
        n = eager.lens.clone()
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        shortened += int((eager.lens < n).sum())
        for a, b in ((eager.out, captured.out), (eager.lens, captured.lens), (eager.tables, captured.tables),
                     (eager.k, captured.k), (eager.v, captured.v), (eager.top, captured.top),
                     (eager.step.scores, captured.step.scores), (eager.step.kept, captured.step.kept)):
            assert torch.equal(a, b), t
        for loop in (eager, captured):
            loop.pos[:2] += 1
    assert shortened >= 6 and eager.step.error_flags() == 0 and captured.step.error_flags() == 0
