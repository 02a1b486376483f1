"""Bounded decode steps whose sequences are shortened between them."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import BoundedDecodeStep
from tests.gpu_helpers import device
from tests.test_gpu_share import i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
LAYERS, B, HQ, HKV, D, WIDTH, NB = 2, 3, 8, 2, 64, 6, 20


class Loop:
    def __init__(self):
        dev = device()
        g = torch.Generator(device=dev).manual_seed(8)
        self.step = BoundedDecodeStep(B, HQ, HKV, D, WIDTH, LAYERS, BF, dev, 40, 44, 2, 10)
        self.k, self.v = (torch.zeros(LAYERS, NB, HKV, 16, D, dtype=BF, device=dev) for _ in range(2))
        self.tables, self.lens = torch.full((B, WIDTH), -1, dtype=torch.int32, device=dev), i32([0, 0, -1])
        self.stack, self.top, self.extra = i32(list(range(NB))), i32([NB]), i32([0] * NB)
        self.pos = i32([0, 0, -1])
        self.x = torch.empty(LAYERS, B, HQ + 2 * HKV, D, dtype=BF, device=dev)
        self.out = torch.zeros(LAYERS, B, HQ, D, dtype=BF, device=dev)
        self.w = torch.ones(D, dtype=BF, device=dev) + 0.1 * torch.randn(D, generator=g, device=dev).to(BF)
        self.table = ops.rope_table(100, D, 1e4, dev)

    def run(self, check=None):
        ops.xs_block_alloc_decode(self.tables, self.lens, self.stack, self.top)
        for l in range(LAYERS):
            before = self.step.scores[l].clone() if check else None
            self.step.run(l, self.out[l], *self.x[l].split([HQ, HKV, HKV], 1), self.w, self.w, self.table, self.pos,
                          self.k[l], self.v[l], self.tables, self.lens, D ** -0.5)
            if check:
                check(l, before)
        self.step.bound(self.k, self.v, self.tables, self.lens, self.stack, self.top, self.extra)

    def cut(self, lens):
        ops.xs_block_truncate(i32(list(range(B))), i32(lens), self.tables, self.lens, self.stack, self.top, self.extra)


def test_replaced_tokens_start_from_zero():
    """Each layer's scores are those of the attention with the scored lengths that a list keeps."""
    loop = Loop()
    g = torch.Generator(device=device()).manual_seed(9)
    ws = ops.BoundedWorkspace(B, HQ, HKV, D, device(), WIDTH)
    scored = [0, 0, 0]

    def check(l, before):
        out = torch.empty_like(loop.out[l])
        ops.xs_paged_decode_weights(out, before, loop.step.q, loop.k[l], loop.v[l], loop.tables, loop.lens, D ** -0.5, ws,
                                    scored_lens=i32(scored))
        assert torch.equal(out, loop.out[l]) and torch.equal(before, loop.step.scores[l]), (t, l)

    for t in range(70):
        loop.x.copy_(torch.randn(loop.x.shape, generator=g, device=device()))
        if t in (17, 30, 58):       # several tokens back, over a page's end
            n = loop.lens.tolist()
            to = [n[0] - 5, n[1] - (1 if t == 30 else 18 if n[1] > 20 else 9), -1]
            loop.cut(to)
            scored = [min(s, m) if m >= 0 else s for s, m in zip(scored, to)]
        if t == 20:
            loop.lens[2] = 0
        loop.run(check)
        loop.pos[:2] += 1
        if t >= 20:
            loop.pos[2] += 1
        scored = [max(n, 0) for n in loop.lens.tolist()]
    assert loop.step.error_flags() == 0


def test_captured_steps_follow_a_rollback():
    eager, captured = Loop(), Loop()
    g = torch.Generator(device=device()).manual_seed(10)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        captured.run()
    for t in range(60):
        x = torch.randn(eager.x.shape, generator=g, device=device())
        for loop in (eager, captured):
            loop.x.copy_(x)
            if t in (10, 33, 50):
                loop.cut([n - 4 if n > 0 else -1 for n in loop.lens.tolist()])
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in ((eager.out, captured.out), (eager.lens, captured.lens), (eager.tables, captured.tables),
                     (eager.step.scores, captured.step.scores), (eager.step.scored, captured.step.scored)):
            assert torch.equal(a, b), t
        for loop in (eager, captured):
            loop.pos[:2] += 1
