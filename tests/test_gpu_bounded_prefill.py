"""Prompt chunks with first tokens and a window, against 64 bits."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests import plain_bounded as plain
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def chunk(T, start, Hq, Hkv, D, seed, first, window, std=1.0):
    """Pages whose rows that no query sees are NaN (V) and junk (K); unseen pages have no block."""
    g = torch.Generator().manual_seed(seed)
    n = start + T
    pages = -(-n // 16)
    k, v = (torch.randn(pages + 2, Hkv, 16, D, generator=g).to(BF) for _ in range(2))
    ids = torch.randperm(pages + 2, generator=g)[:pages].to(torch.int32)
    low = max(0, start + 1 - window) if window else 0
    seen = [t for t in range(n) if t < first or t >= low]
    unseen = torch.ones(pages + 2, 16, dtype=torch.bool)
    table = torch.full((pages,), -1, dtype=torch.int32)
    for t in seen:
        table[t // 16] = ids[t // 16]
        unseen[int(ids[t // 16]), t % 16] = False
    for x in (k, v):
        x.permute(0, 2, 1, 3)[unseen] = float("nan")
    q = (torch.randn(T, Hq, D, generator=g) * std).to(BF)
    return q, k, v, table


@pytest.mark.parametrize("first,window", [(0, 0), (4, 0), (0, 1), (4, 1), (1, 16), (4, 100), (130, 50), (5, 129), (300, 200),
                                          (4, 5000)])
@pytest.mark.parametrize("T,start,Hq,Hkv,D", [(1, 0, 4, 1, 128), (40, 3, 8, 2, 128), (130, 270, 2, 2, 64), (70, 500, 8, 1, 64),
                                              (200, 129, 4, 2, 128)])
def test_masks(T, start, Hq, Hkv, D, first, window):
    q, k, v, ids = chunk(T, start, Hq, Hkv, D, T + first, first, window)
    dev = device()
    out = torch.full((T, Hq, D), 7.0, dtype=BF, device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ops.xs_paged_prefill_first(out, q.to(dev), k.to(dev), v.to(dev), ids.to(dev), start, D ** -0.5, first=first,
                               window=window, err_flag=err)
    ref, bound = plain.prefill(q, k, v, ids.tolist(), start, D ** -0.5, first, window)
    d = (out.cpu().double() - ref).abs()
    assert bool((d <= bound).all()), f"off by {d.max():.3e}, {(d / bound).max():.2f} of the bound"
    assert int(err) == 0


def test_all_logits_far_below_zero():
    # Rows whose first tile is wholly masked, with logits near -1000 behind it.
    q, k, v, ids = chunk(64, 600, 4, 1, 64, 1, 0, 70, std=0.0)
    q[:] = -16.0
    k = torch.where(k.isnan(), k, 1.0 + 0.01 * k)
    dev = device()
    out = torch.empty(64, 4, 64, dtype=BF, device=dev)
    ops.xs_paged_prefill_first(out, q.to(dev), k.to(dev), v.to(dev), ids.to(dev), 600, 1.0, window=70)
    ref, bound = plain.prefill(q, k, v, ids.tolist(), 600, 1.0, 0, 70)
    assert bool(((out.cpu().double() - ref).abs() <= bound).all())


def test_without_a_window_it_is_the_causal_call():
    q, k, v, ids = (x.to(device()) for x in chunk(300, 77, 8, 2, 128, 5, 0, 0))
    a, b = torch.empty_like(q), torch.empty_like(q)
    ops.xs_paged_prefill_first(a, q, k, v, ids, 77, 0.1, first=9)
    v2 = torch.where(v.isnan(), torch.zeros_like(v), v)
    ops.xs_paged_prefill_tc(b, q, k, v2, ids, 77, 0.1)
    # Their sums may run in different orders (a Q tile's keys in two parts that are
    # joined): each is within `bound` of the exact value, so they are within twice
    # that of one another.
    _, bound = plain.prefill(q.cpu(), k.cpu(), v2.cpu(), ids.tolist(), 77, 0.1, 9, 0)
    assert bool(((a.double() - b.double()).abs().cpu() <= 2 * bound).all())


@pytest.mark.parametrize("T", [400, 640, 1], ids=["pairs", "pairs-and-halves", "one"])
@pytest.mark.parametrize("first,window", [(5, 300), (0, 130), (140, 20)])
def test_more_tiles_than_processors(T, first, window):
    # CTAs of two Q tiles (the last one's second without queries), and of one each in the last wave.
    q, k, v, ids = chunk(T, 500, 64, 8, 64, T, first, window)
    out, err = torch.full((T, 64, 64), 7.0, dtype=BF, device=device()), torch.zeros(1, dtype=torch.int32, device=device())
    x = [y.to(device()) for y in (q, k, v, ids)]
    ref, bound = plain.prefill(q, k, v, ids.tolist(), 500, 0.125, first, window)
    for _ in range(2):
        ops.xs_paged_prefill_first(out, *x, 500, 0.125, first=first, window=window, err_flag=err)
        d = (out.cpu().double() - ref).abs()
        assert bool((d <= bound).all()), f"off by {d.max():.3e}, {(d / bound).max():.2f} of the bound"
    assert int(err) == 0


@pytest.mark.parametrize("start", [0, 63, 64, 127, 191, 192, 255, 320, 447])
def test_few_key_tiles(start):
    # One key tile to four: an even and an odd number of them for the two halves of the softmax.
    q, k, v, ids = chunk(64, start, 8, 1, 128, start, 0, 0, std=3.0)
    out = torch.empty(64, 8, 128, dtype=BF, device=device())
    ops.xs_paged_prefill_first(out, *(y.to(device()) for y in (q, k, v, ids)), start, 0.125)
    ref, bound = plain.prefill(q, k, v, ids.tolist(), start, 0.125, 0, 0)
    d = (out.cpu().double() - ref).abs()
    assert bool((d <= bound).all()), f"off by {d.max():.3e}, {(d / bound).max():.2f} of the bound"


def test_captured_and_a_bad_block():
    q, k, v, ids = (x.to(device()) for x in chunk(100, 300, 4, 2, 64, 6, 4, 90))
    out, err = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device=device())
    run = lambda: ops.xs_paged_prefill_first(out, q, k, v, ids, 300, 0.1, first=4, window=90, err_flag=err)  # noqa: E731
    run()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    out.zero_()
    graph.replay()
    assert torch.equal(out, want) and int(err) == 0
    ids[5] = 1 << 24        # a page that no query sees
    run()
    assert int(err) == 0 and torch.equal(out, want)
    ids[16] = 1 << 24
    run()
    assert int(err) == ops.FLAG_BAD_BLOCK


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 4, 1, 128), (20, 8, 1, 64), (33, 8, 8, 128), (130, 16, 4, 64), (250, 4, 4, 128),
                                        (600, 8, 8, 64)])
@pytest.mark.parametrize("first,window", [(0, 0), (40, 1500), (300, 700), (3, 260)])
def test_keys_shared_by_a_cluster(T, Hq, Hkv, D, first, window):
    # One to 40 Q tiles, with lists of 3 to 25 key tiles in 2 to 8 parts.
    q, k, v, ids = chunk(T, 2317, Hq, Hkv, D, T + window, first, window, std=2.0)
    dev = device()
    out, err = torch.full((T, Hq, D), 7.0, dtype=BF, device=dev), torch.zeros(1, dtype=torch.int32, device=dev)
    x = [y.to(dev) for y in (q, k, v, ids)]
    run = lambda: ops.xs_paged_prefill_first(out, *x, 2317, 0.1, first=first, window=window, err_flag=err)  # noqa: E731
    run()
    ref, bound = plain.prefill(q, k, v, ids.tolist(), 2317, 0.1, first, window)
    d = (out.cpu().double() - ref).abs()
    assert bool((d <= bound).all()), f"off by {d.max():.3e}, {(d / bound).max():.2f} of the bound"
    want = out.clone()
    for _ in range(3):
        out.fill_(7.0)
        run()
        assert torch.equal(out, want), "the same result on every run"
    assert int(err) == 0


def test_infinities_and_nan_that_are_seen():
    # In one part of the keys: they reach the outputs that they concern, through the cluster's join.
    q, k, v, ids = chunk(16, 1500, 4, 2, 64, 9, 0, 0)
    v[int(ids[20]), 0, 3, 7] = float("nan")
    v[int(ids[70]), 1, 0, 5] = float("inf")
    out = torch.empty(16, 4, 64, dtype=BF, device=device())
    ops.xs_paged_prefill_first(out, *(y.to(device()) for y in (q, k, v, ids)), 1500, 0.125)
    out = out.float().cpu()
    assert bool(out[:, :2, 7].isnan().all()) and bool((out[:, 2:, 5] == float("inf")).all())
    rest = torch.ones(16, 4, 64, dtype=torch.bool)
    rest[:, :2, 7] = rest[:, 2:, 5] = False
    v[int(ids[20]), 0, 3, 7] = v[int(ids[70]), 1, 0, 5] = 0
    ref, bound = plain.prefill(q, k, v, ids.tolist(), 1500, 0.125, 0, 0)
    assert bool(((out.double() - ref).abs() <= bound)[rest].all())


def test_streams_and_graphs_of_shared_keys():
    # Two graphs of two calls each, replayed beside each other; a call behind other work.
    xs = [chunk(T, 900, 8, 2, 128, T, 4, 700) for T in (48, 20)]
    dx = [[y.to(device()) for y in x] for x in xs]
    outs = [[torch.zeros_like(x[0]) for _ in range(2)] for x in dx]
    streams, graphs = [torch.cuda.Stream() for _ in xs], []
    torch.cuda.synchronize()
    for x, o, s in zip(dx, outs, streams):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for y in o:
                ops.xs_paged_prefill_first(y, *x, 900, 0.1, first=4, window=700)
        graphs.append(graph)
    refs = [plain.prefill(*x[:3], x[3].tolist(), 900, 0.1, 4, 700) for x in xs]
    for _ in range(3):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for o, (ref, bound) in zip(outs, refs):
            for y in o:
                assert bool(((y.cpu().double() - ref).abs() <= bound).all())
                y.zero_()
    # q is written on the stream just before the call, and out read just behind it.
    x, s, late = dx[0], streams[1], torch.zeros_like(dx[0][0])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        late.copy_(x[0])
        ops.xs_paged_prefill_first(outs[0][0], late, *x[1:], 900, 0.1, first=4, window=700)
        got = outs[0][0] + 0
        late.zero_()
    s.synchronize()
    assert bool(((got.cpu().double() - refs[0][0]).abs() <= refs[0][1]).all())
