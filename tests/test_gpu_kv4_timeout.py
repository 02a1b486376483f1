"""The waits of the 4-bit decode attention, made to run out on purpose.

The debug library leaves out the copies of one page of CTA 0's first warp and
shortens the limit of the waits, so the wait for that page runs out with
nothing in flight for it.  In each form of the call: the flag, the launch back
within milliseconds, NaN for what the CTA had to do with and the usual result
for the rest, and the same workspace fit for the next call."""
import time

import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300 import ops
from tests import plain_ops as plain
from tests.gpu_helpers import device

DEFAULT_LIMIT_NS = 4_000_000_000


def test_host_checks():
    xsbuild.build(), xsbuild.build(debug_bounds=True)
    assert ops.load(xsbuild.LIB_PATH).xs_debug_kv4_wait_injection(1_000_000, 2) == -5    # XS_EUNSUPPORTED
    dbg = ops.load_debug()
    assert dbg.xs_debug_kv4_wait_injection(0, -1) == -2          # XS_ESHAPE: no limit
    assert dbg.xs_debug_kv4_wait_injection(1_000_000, -2) == -2  # XS_ESHAPE: bad page


@pytest.mark.gpu
@pytest.mark.parametrize("lens,width,page", [
    ([3000], None, 1),                      # a cluster for each segment
    ([200], None, 1),                       # one CTA of it
    ([12000], None, 2),                     # pieces for all CTAs
    ([1000] * 9, 63, 2),                    # short segments
    ([120] * 9, 63, 0),                     # short segments, a CTA each
    ([3000] * 30, 200, 6),                  # the line, segments cut
    ([300, 500, 0, 420] * 20, 200, 3),      # the line, whole segments, others behind
], ids=["cluster", "alone", "pieces", "short", "short-alone", "line", "line-whole"])
def test_a_wait_that_runs_out(lens, width, page):
    dev = device()
    xsbuild.build(debug_bounds=True)
    dbg = ops.load_debug()
    prev = ops.use_library(dbg)
    try:
        B, Hkv, G, D = len(lens), 8, 4, 128
        pages = -(-max(lens) // 16)
        g = torch.Generator(device=dev).manual_seed(B)
        x = torch.randn(2, B * pages, Hkv, 16, D, generator=g, device=dev).to(torch.bfloat16)
        kc, vc = plain.pack_pages(x[0], False), plain.pack_pages(x[1], True)
        bt = torch.full((B, width or pages), -1, dtype=torch.int32, device=dev)
        bt[:, :pages] = torch.arange(B * pages, dtype=torch.int32, device=dev).view(B, pages)
        n = torch.tensor(lens, dtype=torch.int32, device=dev)
        q = torch.randn(B, G * Hkv, D, generator=g, device=dev).to(torch.bfloat16)
        ws = ops.Kv4Workspace(B, G * Hkv, Hkv, D, dev)
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        good, out = torch.empty_like(q), torch.empty_like(q)
        ops.xs_kv4_decode(good, q, kc, vc, bt, n, 0.1, ws, err_flag=err)
        torch.cuda.synchronize()
        assert int(err) == 0 and bool(good.isfinite().all())
        ops.xs_debug_kv4_wait_injection(1_000_000, page, lib=dbg)   # 1 ms
        try:
            t0 = time.perf_counter()
            ops.xs_kv4_decode(out, q, kc, vc, bt, n, 0.1, ws, err_flag=err)
            torch.cuda.synchronize()
            elapsed = time.perf_counter() - t0
        finally:
            ops.xs_debug_kv4_wait_injection(DEFAULT_LIMIT_NS, -1, lib=dbg)
        assert int(err) == ops.FLAG_TIMEOUT and elapsed < 1.0
        lost = out.isnan().view(B, Hkv, G * D)
        assert torch.equal(lost.any(-1), lost.all(-1)), "whole KV heads"
        lost = lost.all(-1)
        assert bool(lost.any()) and int(lost.sum()) <= 40, "what one CTA had to do with"
        if B == 1 or len(set(lens)) == 1:
            assert bool(lost[0, 0])
        keep = ~lost[:, :, None].expand(B, Hkv, G * D).reshape(B, Hkv * G, D)
        assert torch.equal(out[keep], good[keep])
        assert int(ws.buf[:4096].count_nonzero()) == 0
        err.zero_()
        ops.xs_kv4_decode(out, q, kc, vc, bt, n, 0.1, ws, err_flag=err)
        assert torch.equal(out, good) and int(err) == 0
        assert ops.xs_debug_bounds_failures(reset=True, lib=dbg) == 0
    finally:
        ops.use_library(prev)
