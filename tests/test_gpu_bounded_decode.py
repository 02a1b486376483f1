"""Decode attention to first tokens and a window, and with accumulated weights,
against 64 bits."""
import random

import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300 import ops
from tests import plain_bounded as plain
from tests.gpu_helpers import device

BF, F32 = torch.bfloat16, torch.float32


class Case:
    """A batch with its pages: lens (0 and negative ones too) of a table `width`
    pages wide; what no query sees is NaN, tables of unseen pages are -1 (not
    with `every`, for lengths that change)."""

    def __init__(self, lens, Hq, Hkv, D, dtype, seed, width=None, first=0, window=0, std=1.0, sinks=False,
                 nan=True, every=False):
        dev, g = device(), torch.Generator().manual_seed(seed)
        B = len(lens)
        pages = [-(-max(n, 0) // 16) for n in lens]
        width = width or max(pages + [1])
        nb = sum(pages) + 3
        self.k, self.v = (torch.randn(nb, Hkv, 16, D, generator=g).to(dtype) for _ in range(2))
        perm = torch.randperm(nb, generator=g).tolist()
        tables = torch.full((B, width), -1, dtype=torch.int32)
        unseen = torch.ones(nb, 16, dtype=torch.bool)
        for b, n in enumerate(lens):
            ids = [perm.pop() for _ in range(pages[b])]
            seen = plain.seen_by(max(n, 0), first, window)
            if every:
                tables[b, :pages[b]] = torch.tensor(ids, dtype=torch.int32)
            for t in seen:
                tables[b, t // 16] = ids[t // 16]
                unseen[ids[t // 16], t % 16] = False
        if nan:
            junk = torch.tensor([float("nan"), float("inf"), -float("inf")])
            for x in (self.k, self.v):
                x.permute(0, 2, 1, 3)[unseen] = junk[torch.randint(0, 3, (1,), generator=g)].to(dtype)
        qkv = (torch.randn(B, Hq + 2 * Hkv, D, generator=g) * std).to(dtype)
        self.q = qkv[:, :Hq]
        self.sinks = torch.randn(Hq, generator=g).to(dtype) if sinks else None
        self.lens = torch.tensor(lens, dtype=torch.int32)
        self.tables, self.first, self.window = tables, first, window
        self.scale = D ** -0.5
        self.d = {n: getattr(self, n).to(dev) for n in ("k", "v", "lens", "tables")}
        self.d["q"] = qkv.to(dev)[:, :Hq]           # a slice of a projection's output
        self.d["sinks"] = None if self.sinks is None else self.sinks.to(dev)
        self.out = torch.full((B, Hq, D), 7.0, dtype=dtype, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.shape = (B, Hq, Hkv, D)

    def workspace(self, weights=False):
        return ops.BoundedWorkspace(*self.shape, device(), self.tables.shape[1] if weights else 0)

    def first_call(self, ws, **kw):
        d = self.d
        ops.xs_paged_decode_first(self.out, d["q"], d["k"], d["v"], d["tables"], d["lens"], self.scale, ws,
                                  first=self.first, window=self.window, sinks=d["sinks"], err_flag=self.err, **kw)
        return self.out

    def weights_call(self, ws, scores, scored=None, **kw):
        d = self.d
        ops.xs_paged_decode_weights(self.out, scores, d["q"], d["k"], d["v"], d["tables"], d["lens"], self.scale, ws,
                                    scored_lens=scored, sinks=d["sinks"], err_flag=self.err, **kw)
        return self.out

    def plain(self):
        return plain.decode(self.q, self.k, self.v, self.tables, self.lens, self.scale, self.first, self.window,
                            self.sinks)


def near(out, ref, bound, what=""):
    d = (out.detach().cpu().double() - ref).abs()
    assert bool((d <= bound).all()), f"{what}: off by {d.max():.3e}, {((d / bound).max()):.2f} of the bound"


def batch(n, hi, seed):
    r = random.Random(seed)
    return [r.choice([0, -1, 1, 15, 16, 17, r.randint(1, hi), r.randint(1, hi), hi]) for _ in range(n)]


MASKS = [(0, 0), (4, 0), (0, 1), (1, 1), (4, 16), (4, 15), (5, 33), (16, 64), (17, 100), (100, 40), (1000, 3), (3, 1000)]


@pytest.mark.gpu
@pytest.mark.parametrize("first,window", MASKS)
@pytest.mark.parametrize("shape", [([1, 2, 16, 17, 250], 8, 2, 128, BF), ([300], 4, 4, 64, BF),
                                   ([0, 129, -1, 64], 16, 2, 64, BF), ([33, 250, 0, 1], 4, 2, 64, F32),
                                   ([70, 16], 8, 1, 128, F32)],
                         ids=["g4", "mha", "g8", "f32", "f32g8"])
def test_masks(first, window, shape):
    lens, Hq, Hkv, D, dtype = shape
    c = Case(lens, Hq, Hkv, D, dtype, 7 * first + window, first=first, window=window, sinks=first == 5)
    ws = c.workspace()
    ref, bound, _ = c.plain()
    near(c.first_call(ws), ref, bound)
    assert int(c.err) == 0


# Clusters of 16 (a wide table), 8, 4, 2; the line with whole and with cut segments.
FORMS = [([2000], 8, 4, 128, 600), ([40, 1300], 8, 4, 128, None), (batch(6, 700, 1), 8, 4, 128, None),
         (batch(14, 400, 2), 16, 4, 64, None), (batch(40, 300, 3), 8, 4, 128, 90), (batch(45, 200, 4), 8, 8, 64, None),
         (batch(300, 70, 5), 8, 1, 64, None), ([900] * 3 + [0, 3] * 40 + [1200, 1] * 2, 4, 2, 128, 130)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS, ids=[f"{len(f[0])}x{f[2]}x{f[3]}" for f in FORMS])
def test_forms(form, dtype):
    lens, Hq, Hkv, D, width = form
    c = Case(lens, Hq, Hkv, D, dtype, len(lens), width=width, first=3, window=500, std=2.0)
    ws = c.workspace()
    ref, bound, _ = c.plain()
    for _ in range(2):              # the workspace is left fit for the next call
        near(c.first_call(ws), ref, bound)
        again = c.out.clone()
    assert torch.equal(c.first_call(ws), again), "the same result on every run"
    assert int(c.err) == 0 and int(ws.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("form", FORMS, ids=[f"{len(f[0])}x{f[2]}x{f[3]}" for f in FORMS])
def test_weights(form, dtype):
    lens, Hq, Hkv, D, width = form
    c = Case(lens, Hq, Hkv, D, dtype, 1 + len(lens), width=width, std=2.0, sinks=len(lens) == 6)
    B, S, G = len(lens), c.tables.shape[1] * 16, Hq // Hkv
    g = torch.Generator().manual_seed(B)
    scores = torch.rand(B, Hkv, S, generator=g)
    scored = torch.tensor([max(n, 0) if b % 3 == 0 else 0 if b % 3 == 1 else max(n - 1, 0) // 2
                           for b, n in enumerate(lens)], dtype=torch.int32)
    for b, n in enumerate(lens):
        scores[b, :, int(scored[b]):] = float("nan")        # what was never scored does not count
    ws, dev = c.workspace(True), device()
    ref, bound, weights = c.plain()
    for counts in (scored, None):
        mine = scores.to(dev)
        if counts is None:
            mine = torch.where(mine.isnan(), 0.25, mine)
        before = mine.clone()
        near(c.weights_call(ws, mine, None if counts is None else counts.to(dev)), ref, bound)
        for b, n in enumerate(lens):
            n, got = max(n, 0), mine[b].cpu().double()
            k = max(n - 1, 0) if counts is None else int(counts[b])
            assert torch.equal(mine[b, :, n:].cpu().nan_to_num(9), before[b, :, n:].cpu().nan_to_num(9)), "behind the length"
            if n == 0:
                continue
            _, p, off = weights[b]
            add = p.view(Hkv, G, n).sum(1)
            old = before[b, :, :n].cpu().double()
            old[:, k:] = 0
            want = old + add
            near(got[:, :n], want, off.view(Hkv, G, n).sum(1) + (G + 2) * 2.0 ** -24 * want + 1e-30, f"scores of {b}")
    assert int(c.err) == 0 and int(ws.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 40], ids=["cluster", "line"])
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
def test_infinities_and_nan_that_are_seen(B, dtype):
    c = Case([200] * B, 4, 2, 64, dtype, 3, first=2, window=150, nan=False)
    k, v, tables = c.d["k"], c.d["v"], c.tables
    at = lambda t: (int(tables[0, t // 16]), t % 16)        # noqa: E731
    (b0, o0), (b1, o1), (b2, o2) = at(199), at(1), at(120)
    v[b0, 0, o0, 5] = float("inf")
    v[b1, 0, o1, 9] = -float("inf")
    v[b2, 1, o2, 0] = float("nan")
    out = c.first_call(c.workspace())[0].float().cpu()
    assert bool((out[:2, 5] == float("inf")).all()) and bool((out[:2, 9] == -float("inf")).all())
    assert bool(out[2:, 0].isnan().all())
    rest = torch.ones(4, 64, dtype=torch.bool)
    rest[:2, 5] = rest[:2, 9] = rest[2:, 0] = False
    ref, bound, _ = c.plain()
    near(out[rest], ref[0][rest], bound[0][rest])
    # A key of infinities: its logit is an infinity of either sign, or NaN.
    k[b2, 1, o2] = 0
    v[b2, 1, o2, 0] = 0
    k[b2, 1, o2, 0] = float("inf")
    out = c.first_call(c.workspace())[0].float().cpu()
    for h in (2, 3):
        if float(c.q[0, h, 0]) > 0:
            assert bool(out[h].isnan().all())
        else:
            c.k, c.v = k.cpu(), v.cpu()
            assert bool(out[h].isfinite().all())


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 40], ids=["cluster", "line"])
def test_far_logits(B):
    # Logits of thousands, and a page of them far below all others.
    c = Case([100] * B, 8, 2, 128, BF, 11, std=400.0, first=1, window=90)
    ref, bound, _ = c.plain()
    near(c.first_call(c.workspace()), ref, bound)
    c = Case([100] * B, 8, 2, 128, BF, 12)
    c.d["k"][int(c.tables[0, 0])] *= 1e30
    c.k = c.d["k"].cpu()
    c.d["q"][0] = c.d["q"][0].abs() * -1
    c.q[0] = c.q[0].abs() * -1
    c.d["k"].abs_(), c.k.abs_()
    ref, bound, _ = c.plain()
    out = c.first_call(c.workspace())
    near(out[1:], ref[1:], bound[1:])
    assert bool(out[0].isfinite().all())


@pytest.mark.gpu
def test_a_head_whose_logits_are_all_minus_infinity():
    c = Case([40], 2, 1, 64, F32, 5, nan=False)
    c.d["k"][..., 0] = float("inf")
    c.d["q"][:, 0, 0] = -1.0
    c.d["q"][:, 1, 0] = 1.0
    out = c.first_call(c.workspace())
    assert bool(out.isnan().all())      # 0 / 0, and infinity - infinity


@pytest.mark.gpu
def test_bad_blocks_and_lengths():
    for B in (2, 60):
        c = Case([50] * B, 4, 2, 64, BF, 2, width=4, nan=False)
        ws = c.workspace()
        good = c.first_call(ws).clone()
        c.d["tables"][1, 1] = 1 << 20
        out = c.first_call(ws)
        assert int(c.err) == ops.FLAG_BAD_BLOCK
        keep = [b for b in range(B) if b != 1]
        assert torch.equal(out[keep], good[keep])
        c.err.zero_()
        c.d["tables"][1, 1] = c.tables[1, 1]
        c.d["tables"][1, 3] = c.tables[1, 0]
        c.d["lens"][1] = 65
        out = c.first_call(ws)
        assert int(c.err) == ops.FLAG_BAD_LEN and torch.equal(out[keep], good[keep])
        scores = torch.zeros(B, 2, 64, device=device())
        c.err.zero_()
        c.weights_call(c.workspace(True), scores)
        assert int(c.err) == ops.FLAG_BAD_LEN
        assert torch.allclose(scores.sum(-1), torch.full((B, 2), 2.0, device=device()), atol=1e-4)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [2, 50], ids=["cluster", "line"])
def test_captured_and_on_other_streams(B):
    # Two captured calls with workspaces of their own, replayed beside each other
    # while lengths change between the replays.
    cases = [Case([90 + 3 * i] * B, 8, 4, 64, BF, 20 + i, first=4, window=60, nan=False, every=True) for i in range(2)]
    ws = [c.workspace() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    graphs = []
    for c, w, s in zip(cases, ws, streams):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.first_call(w)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.first_call(w)
            c.first_call(w)
        graphs.append(graph)
    for n in (90, 17, 1, 64, 0, 77):
        for c in cases:
            c.lens.fill_(n)
            c.d["lens"].fill_(n)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for c in cases:
            ref, bound, _ = c.plain()
            near(c.out, ref, bound, f"length {n}")
    # On a stream that is named, behind work on it.
    c, s = cases[0], streams[1]
    with torch.cuda.stream(s):
        torch.cuda._sleep(1_000_000)
        c.d["lens"].fill_(33)
    c.first_call(ws[0], stream=s)
    s.synchronize()
    c.lens.fill_(33)
    ref, bound, _ = c.plain()
    near(c.out, ref, bound)


@pytest.mark.gpu
def test_long_table_and_offsets_beyond_32_bits():
    # Pools of more than 2^31 elements, pages at both ends.
    dev = device()
    Hkv, D, nb = 8, 128, (1 << 31) // (8 * 16 * 128) + 40
    k = torch.zeros(nb, Hkv, 16, D, dtype=BF, device=dev)
    v = torch.zeros(nb, Hkv, 16, D, dtype=BF, device=dev)
    g = torch.Generator(device=dev).manual_seed(1)
    ids = [nb - 1, 0, nb - 2, 1, nb // 2]
    for i in ids:
        k[i] = torch.randn(Hkv, 16, D, generator=g, device=dev).to(BF)
        v[i] = torch.randn(Hkv, 16, D, generator=g, device=dev).to(BF)
    q = torch.randn(1, 16, D, generator=g, device=dev).to(BF)
    out = torch.empty_like(q)
    tables = torch.full((1, 4096), -1, dtype=torch.int32, device=dev)
    tables[0, :5] = torch.tensor(ids, dtype=torch.int32, device=dev)
    lens = torch.tensor([75], dtype=torch.int32, device=dev)
    ws = ops.BoundedWorkspace(1, 16, Hkv, D, dev, 4096)
    small = torch.tensor([[0, 1, 2, 3, 4]], dtype=torch.int32)
    ref, bound, weights = plain.decode(q.cpu(), k[ids].cpu(), v[ids].cpu(), small, lens.cpu(), 0.1, 4, 40)
    ops.xs_paged_decode_first(out, q, k, v, tables, lens, 0.1, ws, first=4, window=40)
    near(out, ref, bound)
    ref, bound, weights = plain.decode(q.cpu(), k[ids].cpu(), v[ids].cpu(), small, lens.cpu(), 0.1)
    scores = torch.zeros(1, Hkv, 65536, device=dev)
    ops.xs_paged_decode_weights(out, scores, q, k, v, tables, lens, 0.1, ws)
    near(out, ref, bound)
    assert torch.allclose(scores[0, :, :75].cpu().double(), weights[0][1].view(Hkv, 2, 75).sum(1), atol=1e-5)


@pytest.mark.gpu
def test_a_prompts_last_rows_as_sequences_of_one_table():
    # Several rows of one sequence's table, as the weights of a prompt's end are counted.
    c = Case([60], 4, 2, 64, BF, 8, nan=False)
    dev, R = device(), 5
    g = torch.Generator(device=dev).manual_seed(2)
    q = torch.randn(R, 4, 64, generator=g, device=dev).to(BF)
    tables = c.d["tables"].expand(R, -1).contiguous()
    lens = torch.arange(56, 61, dtype=torch.int32, device=dev)
    scores, out = torch.full((R, 2, 64), 5.0, device=dev), torch.empty_like(q)
    ws = ops.BoundedWorkspace(R, 4, 2, 64, dev, 4)
    ops.xs_paged_decode_weights(out, scores, q, c.d["k"], c.d["v"], tables, lens, c.scale, ws,
                                scored_lens=torch.zeros(R, dtype=torch.int32, device=dev))
    ref, bound, weights = plain.decode(q.cpu(), c.k, c.v, tables.cpu(), lens.cpu(), c.scale)
    near(out, ref, bound)
    for r in range(R):
        n = 56 + r
        assert torch.allclose(scores[r, :, :n].cpu().double(), weights[r][1].view(2, 2, n).sum(1), atol=1e-5)
        assert bool((scores[r, :, n:] == 5.0).all())


def test_wait_injection_host_checks():
    xsbuild.build(), xsbuild.build(debug_bounds=True)
    assert ops.load(xsbuild.LIB_PATH).xs_debug_bounded_wait_injection(1_000_000, 2) == -5
    dbg = ops.load_debug()
    assert dbg.xs_debug_bounded_wait_injection(0, -1) == -2
    assert dbg.xs_debug_bounded_wait_injection(1_000_000, -2) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [False, True], ids=["first", "weights"])
@pytest.mark.parametrize("lens,page", [([3000], 1), ([200] * 9, 0), ([1000] * 30, 6), ([100, 0, 130] * 20, 1),
                                        ([3000, 17] * 30, 2)],
                         ids=["cluster", "cluster-short", "segments", "segments-short", "line"])
def test_a_wait_that_runs_out(lens, page, weights):
    # A page of CTA 0's first warp is left out: nothing is in flight for it.
    dev = device()
    xsbuild.build(debug_bounds=True)
    dbg = ops.load_debug()
    prev = ops.use_library(dbg)
    try:
        c = Case(lens, 32, 8, 128, BF, 4)
        ws = c.workspace(weights)
        scores = torch.zeros(len(lens), 8, c.tables.shape[1] * 16, device=dev)
        call = (lambda: c.weights_call(ws, scores)) if weights else (lambda: c.first_call(ws))
        good = call().clone()
        assert int(c.err) == 0 and bool(good.isfinite().all())
        ops.xs_debug_bounded_wait_injection(1_000_000, page, lib=dbg)   # 1 ms
        try:
            out = call().clone()
            torch.cuda.synchronize()
        finally:
            ops.xs_debug_bounded_wait_injection(4_000_000_000, -1, lib=dbg)
        assert int(c.err) == ops.FLAG_TIMEOUT
        lost = out.isnan().view(len(lens), 8, 4 * 128)
        assert torch.equal(lost.any(-1), lost.all(-1)), "whole KV heads"
        lost = lost.all(-1)
        assert 0 < int(lost.sum()) <= 12, "what one warp had to do with"
        keep = ~lost[:, :, None].expand(len(lens), 8, 512).reshape(out.shape)
        assert torch.equal(out[keep], good[keep])
        c.err.zero_()
        assert torch.equal(call(), good) and int(c.err) == 0
        assert ops.xs_debug_bounds_failures(reset=True, lib=dbg) == 0
    finally:
        ops.use_library(prev)


@pytest.mark.gpu
@pytest.mark.parametrize("weights", [False, True], ids=["first", "weights"])
def test_a_very_large_batch(weights):
    # More sequences than a CTA for each segment looks at; one long among short ones.
    lens = [(37 * i) % 45 - 3 for i in range(600)]
    lens[311] = 900
    c = Case(lens, 2, 2, 64, BF, 77, first=0 if weights else 2, window=0 if weights else 600)
    ws = c.workspace(weights)
    ref, bound, w = c.plain()
    scores = torch.zeros(600, 2, c.tables.shape[1] * 16, device=device())
    for _ in range(2):
        near(c.weights_call(ws, scores, torch.zeros(600, dtype=torch.int32, device=device())) if weights
             else c.first_call(ws), ref, bound)
    if weights:
        for b, n in enumerate(lens):
            if n > 0:
                near(scores[b, :, :n], w[b][1], w[b][2] + 2.0 ** -22 * w[b][1] + 1e-30)
    assert int(c.err) == 0 and int(ws.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1200] + [20] * 19, [300] * 20, [16] * 150, [40, 80] * 30 + [2500]],
                         ids=["line-long", "segments", "short", "line"])
def test_forms_of_many_segments(lens):
    # Both forms of the kernel for many segments, one after the other on one workspace.
    cs = [Case(x, 16, 8, 64, BF, len(x), width=160) for x in (lens, [100] * len(lens))]
    ws = cs[0].workspace(True)
    for c in cs * 2:
        ref, bound, w = c.plain()
        scores = torch.zeros(len(lens), 8, 2560, device=device())
        near(c.weights_call(ws, scores), ref, bound)
        for b in (0, len(lens) // 2, len(lens) - 1):
            n = int(c.lens[b])
            want, off = w[b][1].view(8, 2, n).sum(1), w[b][2].view(8, 2, n).sum(1)
            near(scores[b, :, :n], want, off + 2.0 ** -22 * want + 1e-30)
        near(c.first_call(ws), ref, bound)
        assert int(ws.buf[:5120].count_nonzero()) == 0


def check_scores(c, scores, weights, G, b, what=""):
    n = max(int(c.lens[b]), 0)
    if n:
        want, off = weights[b][1].view(-1, G, n).sum(1), weights[b][2].view(-1, G, n).sum(1)
        near(scores[b, :, :n], want, off + (G + 2) * 2.0 ** -24 * want + 1e-30, f"scores of {b} {what}")


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lens,Hq,Hkv", [([9001, 3], 8, 1), ([2000, 1999] * 40, 8, 1), ([1500] * 118 + [17, 900], 16, 2)],
                         ids=["cluster", "cta", "segments"])
def test_weights_of_more_logits_than_shared_memory_holds(lens, Hq, Hkv, dtype):
    c = Case(lens, Hq, Hkv, 64, dtype, len(lens))
    ws, scores = c.workspace(True), torch.full((len(lens), Hkv, c.tables.shape[1] * 16), 3.0, device=device())
    scored = torch.zeros(len(lens), dtype=torch.int32, device=device())
    ref, bound, w = c.plain()
    for _ in range(2):
        near(c.weights_call(ws, scores, scored), ref, bound)
        for b, n in enumerate(lens):
            check_scores(c, scores, w, Hq // Hkv, b)
            assert bool((scores[b, :, n:] == 3.0).all())
    assert int(c.err) == 0 and int(ws.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("B", [2, 50], ids=["cluster", "many"])
def test_weights_captured_beside_each_other(B):
    # Two graphs of two calls each, on streams and workspaces of their own; between
    # the replays lengths of one size (a CTA for each segment, where there are many)
    # change to unlike ones (the line) and back.
    cases = [Case([600] * B, 8, 4, 64, BF, 30 + i, width=150, nan=False, every=True) for i in range(2)]
    ws = [c.workspace(True) for c in cases]
    scores = [torch.zeros(B, 4, 2400, device=device()) for _ in cases]
    scored = [torch.zeros(B, dtype=torch.int32, device=device()) for _ in cases]
    streams, graphs = [torch.cuda.Stream() for _ in cases], []
    torch.cuda.synchronize()
    for c, w, x, n, s in zip(cases, ws, scores, scored, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            c.weights_call(w, x, n)
            c.weights_call(w, x, c.d["lens"])       # (every token has a score now)
        graphs.append(graph)
    r = random.Random(B)
    for kind in ("same", "unlike", "short", "unlike", "same"):
        for c in cases:
            lens = [{"same": 600 - b % 5, "unlike": r.choice([1, 5, 40]), "short": 20}[kind] for b in range(B)]
            if kind == "unlike":
                lens[r.randrange(B)], lens[0] = 590, 0
            c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
            c.d["lens"].copy_(c.lens)
        torch.cuda.synchronize()
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for c, x, w in zip(cases, scores, ws):
            ref, bound, weights = c.plain()
            near(c.out, ref, bound, kind)
            for b in range(B):
                check_scores(c, x / 2, weights, 2, b, kind)
            assert int(c.err) == 0 and int(w.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
def test_a_workspace_serves_smaller_calls():
    ws = ops.BoundedWorkspace(64, 8, 4, 64, device(), 200)
    for lens, width in (([700] * 60, 60), ([30, 900], 200), ([100, 1] * 25, 10), ([900] + [10] * 63, 200)):
        c = Case(lens, 8, 4, 64, BF, len(lens), width=width)
        scores = torch.zeros(len(lens), 4, width * 16, device=device())
        ref, bound, w = c.plain()
        near(c.weights_call(ws, scores), ref, bound)
        for b in range(len(lens)):
            check_scores(c, scores, w, 2, b)
        near(c.first_call(ws), ref, bound)
        assert int(ws.buf[:5120].count_nonzero()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[40] * 280, [700] + [3] * 279, [64] * 256, [1] * 257 + [2000] * 40], ids=["same", "one-long", "256", "long-last"])
def test_weights_at_the_forms_limits(lens):
    # Batches about as large as a CTA for each segment is given to, of one KV head.
    c = Case(lens, 4, 1, 64, BF, len(lens), width=130)
    ws, scores = c.workspace(True), torch.zeros(len(lens), 1, 2080, device=device())
    ref, bound, w = c.plain()
    for _ in range(2):
        near(c.weights_call(ws, scores, torch.zeros(len(lens), dtype=torch.int32, device=device())), ref, bound)
        for b in range(0, len(lens), 7):
            check_scores(c, scores, w, 4, b)
        check_scores(c, scores, w, 4, len(lens) - 1)
    assert int(c.err) == 0 and int(ws.buf[:5120].count_nonzero()) == 0
