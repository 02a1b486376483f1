"""What may follow the overlapped launches of a chunked prefill: a call behind
them comes after all of them, the attention that an append ran beside among
them, whether it is captured or not."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("last", ["append", "one token"])
@pytest.mark.parametrize("call", ["norm + rotation", "copy", "read back", "compact and copy"])
def test_calls_behind_overlapped_chunks(call, last, captured):
    """A long chunk's attention, then the next chunk's append (and a short
    attention), then a call that overwrites what the long one reads."""
    dev = device()
    Hq, Hkv, D, n0, T = 32, 8, 128, 6000, 1024
    pages = (n0 + T + 1 + 15) // 16
    nb = 2 * pages
    g = torch.Generator(device=dev).manual_seed(1)
    pools0 = torch.randn(2, 1, nb, Hkv, 16, D, generator=g, device=dev).to(BF)
    pools, ids = torch.empty_like(pools0), torch.arange(pages, nb, dtype=torch.int32, device=dev)
    q0 = torch.randn(T + 1, Hq, D, generator=g, device=dev).to(BF)
    q = torch.empty_like(q0)
    kv = torch.randn(2, 2, Hkv, T, D, generator=g, device=dev).to(BF)
    kv1 = kv[:, 1, :, :1].contiguous()
    out = torch.empty(T + 1, Hq, D, dtype=BF, device=dev)
    junk = torch.randn(T, Hkv, D, generator=g, device=dev).to(BF)
    tab = ops.rope_table(T, D, 1e4, dev)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    pairs = torch.stack([torch.arange(pages, device=dev), torch.arange(pages, nb, device=dev)], 1)
    k4, v4 = ops.kv4_pools(pages, Hkv, D, dev)

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    lens, extra, stack, top = i32([16 * pages]), i32([0] * nb), i32([0] * nb), i32([0])
    remap, moves, count = i32([0] * nb), torch.empty(nb // 2, 2, dtype=torch.int64, device=dev), i32([0])
    tables = torch.empty(1, pages, dtype=torch.int32, device=dev)

    def before():
        pools.copy_(pools0), q.copy_(q0), out.fill_(7.0), lens.fill_(16 * pages)
        tables.copy_(ids[None])

    def prefill(overlap):
        k, v = pools[0, 0], pools[1, 0]
        ops.xs_prefill_append(kv[0, 0], kv[1, 0], k, v, ids, n0, overlap=overlap)
        ops.xs_paged_prefill_tc(out[:T], q[:T], k, v, ids, n0, 0.09, overlap=overlap)
        ops.xs_prefill_append(kv1[0], kv1[1], k, v, ids, n0 + T, overlap=overlap)
        if last == "one token":
            ops.xs_paged_prefill_tc(out[T:], q[T:], k, v, ids, n0 + T, 0.09, overlap=overlap)

    def behind():
        if call == "norm + rotation":
            ops.xs_qk_norm_rope(q[:T], junk, q[:T], junk, None, None, 1e-6, tab, pos)
        elif call == "copy":
            ops.xs_block_copy(pools[0], pools[1], pairs)
        elif call == "read back":
            ops.xs_kv4_unpack(pools[0, 0, pages:], pools[1, 0, pages:], k4, v4, pos[:pages])
        else:
            ops.xs_block_compact(tables, tables, lens, extra, extra, stack, top, remap, moves, count)
            ops.xs_block_copy(pools[0], pools[1], moves, count=count)

    before(), prefill(False)
    torch.cuda.synchronize()
    want = out.clone()
    behind()
    torch.cuda.synchronize()
    want_pools, want_q = pools.clone(), q.clone()

    def all_of_it():
        before(), prefill(True), behind()

    run = all_of_it
    if captured:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            all_of_it()
        torch.cuda.current_stream().wait_stream(s)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            all_of_it()
        run = graph.replay
    for _ in range(10):
        out.zero_(), pools.zero_()
        run()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        # (junk is rotated again by each call, pools and q start anew)
        assert torch.equal(pools, want_pools) and torch.equal(q, want_q)
