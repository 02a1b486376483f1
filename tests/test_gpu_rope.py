"""xs_qk_norm_rope and its two appending forms against 64 bits."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests import plain_ops as plain
from tests.gpu_helpers import device, int_view

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def inputs(T, Hq, Hkv, D, dtype, seed, norm=True, wide=0):
    """q, k, v as slices of one projection's output with `wide` more columns."""
    dev = device()
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(T, (Hq + 2 * Hkv) * D + wide, generator=g, device=dev).to(dtype)
    q = x[:, :Hq * D].view(T, Hq, D)
    k = x[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    v = x[:, (Hq + Hkv) * D:(Hq + 2 * Hkv) * D].view(T, Hkv, D)
    w = [(1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dtype) if norm else None
         for _ in range(2)]
    return x, q, k, v, w[0], w[1]


def table(rows, rot):
    return ops.rope_table(rows, rot, 1e6, device()) if rot else None


def check_rows(out, x, w, eps, tab, pos, rot, inter, what):
    ref, mag = plain.norm_rope(x, w, eps, tab, pos, rot, inter)
    if w is None and not rot:
        assert torch.equal(int_view(out.contiguous()), int_view(x.contiguous())), what
        return
    plain.check(out, ref, plain.norm_rope_bound(ref, mag, x.dtype), what)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,norm", [
    (1, 1, 1, 64, 64, False, True), (1, 32, 8, 128, 128, False, True),
    (7, 12, 12, 64, 32, True, True), (33, 6, 2, 128, 48, False, True),
    (5, 8, 1, 128, 16, True, True), (130, 3, 3, 64, 16, False, False),
    (9, 5, 5, 128, 0, False, True), (3, 2, 1, 64, 0, False, False),
    (257, 32, 8, 128, 128, True, True), (64, 7, 7, 64, 48, True, False),
])
def test_rows(T, Hq, Hkv, D, rot, inter, norm, dtype):
    _, q, k, _, qw, kw = inputs(T, Hq, Hkv, D, dtype, seed=T * 7 + D, norm=norm, wide=64)
    rows = 5000
    tab = table(rows, rot)
    pos = torch.randint(0, rows, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32)
    pos[0], pos[-1] = 0, rows - 1
    pos = pos.to(device())
    err = torch.zeros(1, dtype=torch.int32, device=device())
    qo = torch.empty(T, Hq, D, dtype=dtype, device=device())
    ko = torch.empty(T, Hkv, D, dtype=dtype, device=device())
    ops.xs_qk_norm_rope(qo, ko, q, k, qw, kw, 1e-6, tab, pos, interleaved=inter, err_flag=err)
    check_rows(qo, q, qw, 1e-6, tab, pos, rot, inter, "q")
    check_rows(ko, k, kw, 1e-6, tab, pos, rot, inter, "k")
    assert int(err) == 0


def test_in_place_and_skipped_rows():
    # q_out is q and k_out is k; a negative position leaves its row, one
    # behind the table too, with a flag.
    dev = device()
    g = torch.Generator(device=dev).manual_seed(3)
    q = torch.randn(6, 8, 128, generator=g, device=dev).to(BF)
    k = torch.randn(6, 2, 128, generator=g, device=dev).to(BF)
    tab = table(100, 128)
    pos = torch.tensor([5, -1, 99, 100, 0, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    q0, k0 = q.clone(), k.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ops.xs_qk_norm_rope(q, k, q, k, None, None, 0.0, tab, pos, err_flag=err)
    on = torch.tensor([0, 2, 4], device=dev)
    for got, was in ((q, q0), (k, k0)):
        check_rows(got[on], was[on], None, 0.0, tab, pos[on], 128, False, "in place")
        off = torch.tensor([1, 3, 5], device=dev)
        assert torch.equal(got[off], was[off])
    assert int(err) == ops.FLAG_BAD_LEN


def test_zero_tiny_and_large_rows():
    # A row of zeros stays zero (eps keeps the root finite); rows at both ends
    # of the type's range; one with an infinity and one with a NaN poison
    # themselves only.
    dev = device()
    q = torch.ones(6, 1, 64, device=dev)
    q[0] = 0
    q[1] *= 1e-18
    q[2] *= 3e18
    q[3, 0, 5] = float("inf")
    q[4, 0, 5] = float("nan")
    q = q.to(BF)
    k = q.clone()
    out, ko = torch.empty_like(q), torch.empty_like(k)
    tab = table(8, 64)
    pos = torch.arange(6, dtype=torch.int32, device=dev)
    w = torch.ones(64, dtype=BF, device=dev)
    ops.xs_qk_norm_rope(out, ko, q, k, w, w, 1e-6, tab, pos)
    assert bool((out[0] == 0).all()) and bool(out[[1, 2, 5]].isfinite().all())
    assert bool(out[4].isnan().all()) and bool(out[3].isnan().any())
    for r in (1, 2, 5):
        check_rows(out[r:r + 1], q[r:r + 1], w, 1e-6, tab, pos[r:r + 1], 64, False, f"row {r}")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter", [(1, 4, 1, 64, 64, False), (37, 8, 2, 128, 128, False),
                                                  (50, 12, 12, 64, 32, True)])
def test_append_equals_separate_calls(T, Hq, Hkv, D, rot, inter, dtype):
    # Bit for bit xs_qk_norm_rope + xs_kv_append; rows that are not appended
    # leave the pools alone.
    dev = device()
    _, q, k, v, qw, kw = inputs(T, Hq, Hkv, D, dtype, seed=11, wide=8 * 16)
    tab = table(300, rot)
    nb = T // 16 + 3
    cpu = torch.Generator().manual_seed(4)
    slots = torch.randperm(nb * 16, generator=cpu)[:T].to(torch.int64)
    if T > 3:
        slots[2] = -1
    slots = slots.to(dev)
    pos = torch.randint(0, 300, (T,), generator=cpu).to(torch.int32).to(dev)
    kc = torch.full((nb, Hkv, 16, D), 7.0, dtype=dtype, device=dev)
    vc = torch.full_like(kc, -7.0)
    kr, vr = kc.clone(), vc.clone()
    qo, qr = (torch.empty(T, Hq, D, dtype=dtype, device=dev) for _ in range(2))
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ops.xs_qk_norm_rope_append(qo, q, k, v, qw, kw, 1e-5, tab, pos, kc, vc, slots,
                               interleaved=inter, err_flag=err)
    ko = torch.empty(T, Hkv, D, dtype=dtype, device=dev)
    ops.xs_qk_norm_rope(qr, ko, q, k, qw, kw, 1e-5, tab, pos, interleaved=inter)
    ops.xs_kv_append(ko, v.contiguous(), kr, vr, slots)
    for a, b in ((qo, qr), (kc, kr), (vc, vr)):
        assert torch.equal(int_view(a), int_view(b))
    assert int(err) == 0


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,D", [(1, 4, 4, 64), (61, 32, 8, 128)])
def test_append_paged_equals_separate_calls(B, Hq, Hkv, D, kv4):
    dev = device()
    _, q, k, v, qw, kw = inputs(B, Hq, Hkv, D, BF, seed=12)
    cpu = torch.Generator().manual_seed(6)
    lens = torch.randint(1, 200, (B,), generator=cpu).to(torch.int32)
    if B > 8:
        lens[3], lens[4], lens[5] = 0, -1, 16
    bt = torch.randperm(B * 13, generator=cpu).to(torch.int32).view(B, 13)
    lens, bt = lens.to(dev), bt.to(dev)
    nb = B * 13
    tab = table(200, D)
    if kv4:
        kc, vc = ops.kv4_pools(nb, Hkv, D, dev)
    else:
        kc, vc = (torch.zeros(nb, Hkv, 16, D, dtype=BF, device=dev) for _ in range(2))
    kr, vr = kc.clone(), vc.clone()
    qo = torch.full((B, Hq, D), 3.0, dtype=BF, device=dev)
    qr = qo.clone()
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    ops.xs_qk_norm_rope_append_paged(qo, q, k, v, qw, kw, 1e-6, tab, kc, vc, bt, lens,
                                     err_flag=err)
    ko = k.contiguous()
    ops.xs_qk_norm_rope(qr, ko, q, k, qw, kw, 1e-6, tab, lens - 1)
    (ops.xs_kv4_append_paged if kv4 else ops.xs_kv_append_paged)(ko, v.contiguous(), kr, vr, bt, lens)
    for a, b in ((qo, qr), (kc, kr), (vc, vr)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert int(err) == 0
    if B > 8:
        assert bool((qo[3:5] == 3.0).all())


def test_append_device_errors():
    # Slots behind the pool, block ids outside it, a position beyond the table:
    # flagged, nothing else written.
    dev = device()
    _, q, k, v, qw, kw = inputs(4, 2, 2, 64, BF, seed=13)
    kc = torch.zeros(5, 2, 16, 64, dtype=BF, device=dev)
    vc = torch.zeros_like(kc)
    qo = torch.empty(4, 2, 64, dtype=BF, device=dev)
    pos = torch.zeros(4, dtype=torch.int32, device=dev)
    slots = torch.tensor([80, 2 ** 40, -5, 79], device=dev)
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    tab = table(64, 64)
    ops.xs_qk_norm_rope_append(qo, q, k, v, qw, kw, 1e-6, tab, pos, kc, vc, slots, err_flag=err)
    assert int(err) == ops.FLAG_BAD_SLOT
    assert kc.view(5, 2, 16, 64).ne(0).any(-1).any(1).nonzero().tolist() == [[4, 15]]
    check_rows(qo, q, qw, 1e-6, tab, pos, 64, False, "q is written all the same")
    kc.zero_(), err.zero_()
    bt = torch.tensor([[5, 0], [-1, 0], [1, 2], [3, 4]], dtype=torch.int32, device=dev)
    lens = torch.tensor([1, 2, 33, 32], dtype=torch.int32, device=dev)
    ops.xs_qk_norm_rope_append_paged(qo, q, k, v, qw, kw, 1e-6, tab, kc, vc, bt, lens, err_flag=err)
    assert int(err) == ops.FLAG_BAD_BLOCK | ops.FLAG_BAD_LEN
    assert kc.ne(0).any(-1).any(1).nonzero().tolist() == [[4, 15]]


def test_stream_and_graph():
    # On a side stream, and captured: a replay reads the inputs of that moment.
    dev = device()
    _, q, k, v, qw, kw = inputs(9, 8, 2, 128, BF, seed=14)
    tab, pos = table(64, 128), torch.arange(9, dtype=torch.int32, device=dev)
    qo, ko = torch.empty(9, 8, 128, dtype=BF, device=dev), torch.empty(9, 2, 128, dtype=BF, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ops.xs_qk_norm_rope(qo, ko, q, k, qw, kw, 1e-6, tab, pos)
    s.synchronize()
    check_rows(qo, q, qw, 1e-6, tab, pos, 128, False, "side stream")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ops.xs_qk_norm_rope(qo, ko, q, k, qw, kw, 1e-6, tab, pos)
    pos.add_(7)
    q.mul_(-1.5)
    graph.replay()
    torch.cuda.synchronize()
    check_rows(qo, q, qw, 1e-6, tab, pos, 128, False, "replay q")
    check_rows(ko, k, kw, 1e-6, tab, pos, 128, False, "replay k")


def test_many_rows_of_one_head_and_wide_strides():
    # More rows than one grid covers at a time is not reachable in a small
    # test; rows far apart are: a token stride of 3 GB / T elements.
    dev = device()
    T, D = 40, 64
    wide = torch.empty(T, 40_000_000, dtype=BF, device=dev)     # 3.2 GB: offsets past 2^31 bytes
    g = torch.Generator(device=dev).manual_seed(5)
    wide[:, :3 * D] = torch.randn(T, 3 * D, generator=g, device=dev).to(BF)
    q, k = wide[:, :D].view(T, 1, D), wide[:, D:2 * D].view(T, 1, D)
    tab, pos = table(64, D), torch.arange(T, dtype=torch.int32, device=dev)
    qo, ko = torch.empty(T, 1, D, dtype=BF, device=dev), torch.empty(T, 1, D, dtype=BF, device=dev)
    ops.xs_qk_norm_rope(qo, ko, q, k, None, None, 1e-6, tab, pos)
    check_rows(qo, q, None, 1e-6, tab, pos, D, False, "q")
    check_rows(ko, k, None, 1e-6, tab, pos, D, False, "k")


@pytest.mark.parametrize("T,Hq,Hkv,D,rot,inter,dtype", [
    (20000, 5, 3, 64, 32, False, BF), (9001, 7, 2, 128, 48, True, BF), (5000, 5, 5, 128, 128, False, F32),
    (12003, 1, 1, 64, 64, False, BF),
])
@pytest.mark.parametrize("cache", ["none", "same", "kv4"])
def test_long_calls_equal_short_ones(T, Hq, Hkv, D, rot, inter, dtype, cache):
    # A long call takes several heads of a token at a time, across the borders
    # between q, k and v; calls of 50 tokens take one.  Bit for bit the same.
    if cache == "kv4" and dtype == F32:
        pytest.skip("4-bit pools take bf16 rows")
    dev = device()
    _, q, k, v, qw, kw = inputs(T, Hq, Hkv, D, dtype, seed=T, wide=64)
    tab = table(T + 5, rot)
    pos = torch.randperm(T + 5, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32).to(dev)
    pos[17] = -1
    nb = T // 16 + 2
    slots = torch.randperm(nb * 16, generator=torch.Generator().manual_seed(T + 1))[:T].to(dev)
    slots[:4000] = slots[:4000].sort().values           # consecutive tokens that share a V pair, and not
    slots[40] = -1
    out = []
    for step in (T, 50):
        qo = torch.zeros(T, Hq, D, dtype=dtype, device=dev)
        if cache == "none":
            kc = vc = torch.zeros(T, Hkv, D, dtype=dtype, device=dev)
        elif cache == "same":
            kc, vc = (torch.zeros(nb, Hkv, 16, D, dtype=dtype, device=dev) for _ in range(2))
        else:
            kc, vc = ops.kv4_pools(nb, Hkv, D, dev)
        for a in range(0, T, step):
            s = slice(a, a + step)
            if cache == "none":
                ops.xs_qk_norm_rope(qo[s], kc[s], q[s], k[s], qw, kw, 1e-6, tab, pos[s], interleaved=inter)
            else:
                ops.xs_qk_norm_rope_append(qo[s], q[s], k[s], v[s], qw, kw, 1e-6, tab, pos[s], kc, vc, slots[s],
                                           interleaved=inter)
        out.append((qo, kc, vc))
    for a, b in zip(*out):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    on = torch.arange(100, device=dev)
    on = on[pos[:100] >= 0]
    check_rows(out[0][0][on], q[on], qw, 1e-6, tab, pos[on], rot, inter, "q")
