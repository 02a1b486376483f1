"""Norm + rotation of rows whose squares leave fp32."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests import plain_ops as plain
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SIZES = [1e25, 1.0, 1e37, 1e-25, 1e-36, 3.0, 1e19, 1e-16, 2e-38, 1e18, 1e-14]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("eps", [0.0, 1e-34, 1e-6, 1e30])
def test_rows_of_any_size(D, eps, dtype):
    # Rows of these sizes next to one another: two or four of them share a warp, so
    # that one is scaled before its squares are taken and its neighbour is not.  One row
    # has a single large value among ordinary ones.
    dev, Hq, Hkv = device(), 3, 2
    T = 3 * len(SIZES) + 1
    g = torch.Generator(device=dev).manual_seed(D)
    size = torch.tensor((SIZES * 3 + [1.0]), device=dev)
    q, k = (torch.randn(T, h, D, generator=g, device=dev) for h in (Hq, Hkv))
    q, k = (x / x.abs().amax(-1, keepdim=True) * size[:, None, None] for x in (q, k))
    q[-1, 0, 7] = 1e30
    q, k = q.to(dtype), k.to(dtype)
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(dtype) for _ in range(2))
    tab, pos = ops.rope_table(T, D, 1e4, dev), torch.arange(T, dtype=torch.int32, device=dev)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    ops.xs_qk_norm_rope(qo, ko, q, k, qw, kw, eps, tab, pos)
    for out, x, w in ((qo, q, qw), (ko, k, kw)):
        ref, mag = plain.norm_rope(x, w, eps, tab, pos, D, False)
        assert bool(ref.isfinite().all()) and bool(out.isfinite().all())
        plain.check(out, ref, plain.norm_rope_bound(ref, mag, dtype), f"eps {eps}")


def test_same_row_in_any_company():
    # A row's result does not depend on what the other rows of its warp need.
    dev, D = device(), 64
    g = torch.Generator(device=dev).manual_seed(1)
    row = torch.randn(1, 1, D, generator=g, device=dev).to(BF)
    tab = ops.rope_table(4, D, 1e4, dev)
    w = torch.ones(D, dtype=BF, device=dev)
    pos = torch.ones(4, dtype=torch.int32, device=dev)
    seen = []
    for other in (1.0, 1e30, 1e-30):
        x = row.expand(4, 1, D).clone()
        x[[0, 2, 3]] *= other
        out, ko = torch.empty_like(x), torch.empty_like(x)
        ops.xs_qk_norm_rope(out, ko, x, x, w, w, 1e-6, tab, pos)
        seen.append(out[1].clone())
    assert torch.equal(seen[0], seen[1]) and torch.equal(seen[0], seen[2])


@pytest.mark.parametrize("T", [70, 9000])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 48), (64, 64), (64, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_4_bit_append_equals_separate_calls(D, rot, inter, T):
    # Bit for bit, pairs of either kind: the rows that the fused call quantises
    # are those that the call without pages writes.
    dev, Hq, Hkv = device(), 5, 3
    g = torch.Generator(device=dev).manual_seed(T + rot)
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device=dev).to(BF)
    q, k, v = (y.view(T, -1, D) for y in x.split([Hq * D, Hkv * D, Hkv * D], 1))
    qw, kw = ((1 + 0.2 * torch.randn(D, generator=g, device=dev)).to(BF) for _ in range(2))
    tab, pos = ops.rope_table(T, rot, 1e6, dev), torch.randperm(T, device=dev).to(torch.int32)
    nb = T // 16 + 1
    slots = torch.randperm(nb * 16, generator=torch.Generator().manual_seed(T))[:T].to(dev)
    kc, vc = ops.kv4_pools(nb, Hkv, D, dev)
    kr, vr = ops.kv4_pools(nb, Hkv, D, dev)
    qo, qr = (torch.empty(T, Hq, D, dtype=BF, device=dev) for _ in range(2))
    ko = torch.empty(T, Hkv, D, dtype=BF, device=dev)
    ops.xs_qk_norm_rope_append(qo, q, k, v, qw, kw, 1e-6, tab, pos, kc, vc, slots, interleaved=inter)
    ops.xs_qk_norm_rope(qr, ko, q, k, qw, kw, 1e-6, tab, pos, interleaved=inter)
    ops.xs_kv4_append(ko, v, kr, vr, slots)
    assert torch.equal(qo.view(torch.int16), qr.view(torch.int16))
    assert torch.equal(kc, kr) and torch.equal(vc, vr)
