"""Decode attention over a 4-bit cache: what its weights are rounded to, and
values at the ends of their types."""
import math

import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import Kv4DecodeStep
from tests import plain_ops as plain
from tests.gpu_helpers import device

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def gen(seed):
    return torch.Generator(device=device()).manual_seed(seed)


def pages_of(rows, is_v):
    """Rows [B, pages, Hkv, 16, D] as a pool with the pages in order."""
    return plain.pack_pages(rows.flatten(0, 1).to(BF), is_v)


def tables_of(B, pages, width=None):
    t = torch.full((B, width or pages), -1, dtype=torch.int32, device=device())
    t[:, :pages] = torch.arange(B * pages, dtype=torch.int32, device=device()).view(B, pages)
    return t


def attend_fine(q, kc, vc, pages, lens, scale, sinks=None, window=0):
    """(out, bound) in fp64 where the weights are not rounded to 8 bits.

    The bound: a logit is an fp32 sum of exact products s n q and -8 s q, 34
    additions to a group of 32, each off by at most 2^-22 of the magnitudes
    that meet in it (matrix instructions may cut where fp32 would round),
    which changes a weight by that amount; the exponential and its argument
    add 2^-21 of the logit's size and 2^-21.  A weight times its scale is a
    sum of two bf16 values, of which the second is off by half a step of a
    step: 2^-16.  It enters a sum of up to 64 additions, cut at 2^-22 each:
    2^-16.  The sum of the weights, the join and the division add under
    2^-18.  So 2^-14 of the magnitudes in all, and the output is rounded once
    (2^-8)."""
    B, Hq, D = q.shape
    Hkv = kc.shape[1]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    for b, n in enumerate(lens):
        if n <= 0:
            continue
        a = max(0, n - window) if window else 0
        k, v = (plain.page_values(p[b * pages:b * pages + pages], D, is_v).transpose(0, 1).flatten(1, 2)[:, a:n]
                for p, is_v in ((kc, False), (vc, True)))                # [Hkv, n, D]
        qd = q[b].double().view(Hkv, Hq // Hkv, D)
        x = qd @ k.transpose(1, 2) * scale
        m = x.amax(-1, keepdim=True)
        z = None
        if sinks is not None:
            z = sinks.double().view(Hkv, Hq // Hkv, 1)
            m = torch.maximum(m, z)
        p = torch.exp(x - m)
        w = p / (p.sum(-1, keepdim=True) + (torch.exp(z - m) if z is not None else 0))
        out[b] = (w @ v).view(Hq, D)
        s = k.abs().reshape(*k.shape[:-1], -1, 32).amax(-1) / 7
        sq = qd.abs().reshape(Hkv, Hq // Hkv, -1, 32).sum(-1)
        size = abs(scale) * 23 * (sq @ s.transpose(1, 2))
        off = 34 * 2.0 ** -22 * size + 2.0 ** -21 * (x - m).abs() + 2.0 ** -21
        off = off + (w * off).sum(-1, keepdim=True)
        mag = w @ v.abs()
        bound[b] = ((w * off) @ v.abs() + 2.0 ** -14 * mag).view(Hq, D) + 2.0 ** -8 * out[b].abs() + 1e-37
    return out, bound


def decode(q, kc, vc, bt, lens, scale, sinks=None, window=0):
    ws = ops.Kv4Workspace(q.shape[0], q.shape[1], kc.shape[1], q.shape[2], q.device)
    out = torch.full_like(q, 5.0)
    err = torch.zeros(1, dtype=torch.int32, device=q.device)
    ops.xs_kv4_decode(out, q, kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device=q.device), scale, ws,
                      sinks=sinks, window=window, err_flag=err)
    assert int(err) == 0
    return out


@pytest.mark.parametrize("lens,width,Hkv,G,D", [
    ([500], None, 2, 4, 128),                       # one cluster
    ([490, 3, 17], 900, 8, 1, 64),                  # few sequences under a wide table
    ([1000] * 9, 63, 8, 8, 128),                    # short segments
    ([400, 513, 0, 33] * 12, 200, 8, 4, 128),       # the line
    ([16 * 40 + 7] * 40, 300, 8, 2, 64),            # the line, segments cut
])
@pytest.mark.parametrize("sinks,window", [(False, 0), (True, 290)])
def test_weights_are_not_rounded_to_8_bits(lens, width, Hkv, G, D, sinks, window):
    # Many tokens of like weight: the output is far smaller than what it is
    # summed from, so that a rounding of the weights shows beside its own.
    B, pages = len(lens), -(-max(lens) // 16)
    k, v = (torch.randn(B, pages, Hkv, 16, D, generator=gen(i + B), device=device()) for i in (1, 2))
    kc, vc = pages_of(k, False), pages_of(v, True)
    q = torch.randn(B, G * Hkv, D, generator=gen(3), device=device()).to(BF)
    z = torch.randn(G * Hkv, generator=gen(4), device=device()).to(BF) if sinks else None
    scale = 0.5 / math.sqrt(D)
    out = decode(q, kc, vc, tables_of(B, pages, width), lens, scale, z, window)
    ref, bound = attend_fine(q, kc, vc, pages, lens, scale, z, window)
    plain.check(out, ref, bound)


FORMS = [(1, None), (1, 2000), (9, 100), (70, 2000)]     # (sequences, table width): few, few, short, the line


@pytest.mark.parametrize("B,width", FORMS)
def test_values_near_the_end_of_bf16(B, width):
    # Each group of V holds 3 2^122 (a scale of 3 2^119), and the logits of the
    # second half are 7.9 powers of two above those of the first: a weight
    # above 1 times the scale would be infinite.  As xs_paged_decode_sinks, whose
    # weights are at most 1.
    dev, D, Hkv, G, pages = device(), 128, 8, 2, 16
    k = torch.zeros(B, pages, Hkv, 16, D, device=dev)
    k[:, pages // 2:, ..., 0] = 7.9 * math.log(2.0)
    v = torch.randn(B, pages, Hkv, 16, D, generator=gen(1), device=dev).clamp(-2, 2) * 2.0 ** 120
    sign = torch.randint(0, 2, (B, pages, Hkv, 16, 4), generator=gen(2), device=dev) * 2.0 - 1
    v[..., 5::32] = sign * 3 * 2.0 ** 122
    kc, vc = pages_of(k, False), pages_of(v, True)
    q = torch.zeros(B, G * Hkv, D, dtype=BF, device=dev)
    q[..., 0] = 1
    lens = [16 * pages] * B
    out = decode(q, kc, vc, tables_of(B, pages, width), lens, 1.0)
    assert bool(out.isfinite().all())
    ref, bound = attend_fine(q, kc, vc, pages, lens, 1.0)
    plain.check(out, ref, bound)


@pytest.mark.parametrize("e", [-100, -60, 60, 110])
def test_values_of_any_magnitude(e):
    dev, D, Hkv, G, lens = device(), 64, 2, 4, [700, 45, 16]
    k, v = (torch.randn(3, 44, Hkv, 16, D, generator=gen(i), device=dev) for i in (5, 6))
    kc, vc = pages_of(k, False), pages_of(v * 2.0 ** e, True)
    q = torch.randn(3, G * Hkv, D, generator=gen(7), device=dev).to(BF)
    out = decode(q, kc, vc, tables_of(3, 44), lens, 0.2)
    ref, bound = attend_fine(q, kc, vc, 44, lens, 0.2)
    plain.check(out, ref, bound)


@pytest.mark.parametrize("pages", [2, 16, 40])
@pytest.mark.parametrize("B,width", FORMS)
def test_logits_of_minus_infinity_beside_very_low_ones(B, width, pages):
    # Logits below fp32 in the first half's pages, of -1024 or a little less in
    # the second's: the softmax is that of the second.
    dev, D, Hkv, G = device(), 64, 8, 1
    k = torch.zeros(B, pages, Hkv, 16, D, device=dev)
    k[:, :pages // 2, ..., 0] = -2.0 ** 100
    k[:, pages // 2:, ..., 0] = -2.0 ** -50
    k[:, -1, :, 3, 0] = -(2.0 ** -50 + 2.0 ** -57)
    v = torch.randn(B, pages, Hkv, 16, D, generator=gen(3), device=dev)
    kc, vc = pages_of(k, False), pages_of(v, True)
    q = torch.zeros(B, G * Hkv, D, dtype=BF, device=dev)
    q[..., 0] = 2.0 ** 60
    q[:, 1, 0] = -2.0 ** -60         # a head with ordinary logits beside it
    lens = [16 * pages - 1] * B
    out = decode(q, kc, vc, tables_of(B, pages, width), lens, 1.0)
    assert bool(out.isfinite().all())
    mean = plain.page_values(vc, D, True).view(B, pages, Hkv, 16, D)
    low = mean[:, pages // 2:].transpose(1, 2).flatten(2, 3)[:, :, :-1]       # [B, Hkv, n, D]
    w = torch.ones(low.shape[2], dtype=torch.float64, device=dev)
    w[low.shape[2] - 15 + 3] = math.exp(-8.0)
    ref = (low * (w / w.sum())[:, None]).sum(2)
    mag = (low.abs() * (w / w.sum())[:, None]).sum(2)
    others = [0, 2, 3, 4, 5, 6, 7]
    # (logits of 2^10.5 to 2^-22 of their size: 2^-11.5)
    plain.check(out[:, others], ref[:, others], (2.0 ** -8 * ref.abs() + 2.0 ** -10 * mag)[:, others])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("B,width", FORMS)
def test_infinite_key_is_nan_whatever_the_query(B, width, bad):
    # Queries whose products do not sum exactly: a group with an infinity
    # stands for NaN, and so does its logit.
    dev, D, Hkv, G, pages = device(), 64, 8, 8, 3
    k, v = (torch.randn(B, pages, Hkv, 16, D, generator=gen(i), device=dev) for i in (1, 2))
    kc, vc = pages_of(k, False), pages_of(v, True)
    row = torch.ones(1, Hkv, D, dtype=BF, device=dev)
    row[0, 3, 7] = bad
    ops.xs_kv4_append(row, row * 0, kc, vc, torch.tensor([16 + 5], device=dev))    # token 21 of sequence 0
    q = 2.0 ** -14 * (1 + torch.rand(B, G * Hkv, D, generator=gen(3), device=dev))
    q[..., 0::32] = 1
    q[:, 1::2] *= -1
    out = decode(q.to(BF), kc, vc, tables_of(B, pages, width), [40] * B, 0.5)
    want = torch.zeros_like(out, dtype=torch.bool)
    want[0, 3 * G:4 * G] = True
    assert torch.equal(out.isnan(), want) and bool(out[~want].isfinite().all())


def test_position_behind_the_rotation_table():
    """A sequence longer than the table of cosines and sines: its row of the
    step is neither rotated nor appended, and its output is NaN, not what an
    earlier call's query gives.  The others are as ever."""
    dev, B, Hq, Hkv, D, nb = device(), 4, 8, 2, 128, 40
    tab = ops.rope_table(40, D, 1e4, dev)
    kc, vc = ops.kv4_pools(nb, Hkv, D, dev)
    bt = torch.arange(nb, dtype=torch.int32, device=dev).view(B, 10)
    x = torch.randn(2, B, Hq + 2 * Hkv, D, generator=gen(1), device=dev).to(BF)
    step, alone = Kv4DecodeStep(B, Hq, Hkv, D, dev), Kv4DecodeStep(B, Hq, Hkv, D, dev)
    lens = torch.tensor([39, 40, 1, 0], dtype=torch.int32, device=dev)
    out = torch.empty(B, Hq, D, dtype=BF, device=dev)

    def run(s, i):
        q, k, v = x[i].split([Hq, Hkv, Hkv], 1)
        s.run(out, q, k, v, None, None, tab, kc, vc, bt, lens, 0.1)

    run(step, 0)
    assert step.error_flags() == 0 and bool((out[3] == 0).all()) and bool(out.isfinite().all())
    lens += 1                                              # sequence 1's position is 40
    before = kc.clone(), vc.clone()
    run(step, 1)
    assert step.error_flags() == ops.FLAG_BAD_LEN
    assert bool(out[1].isnan().all()) and bool(out[[0, 2, 3]].isfinite().all())
    for pool, was in zip((kc, vc), before):                # nothing of sequence 1's new row
        assert torch.equal(pool[10:20], was[10:20])
    got = out.clone()
    lens[1] = -1
    run(alone, 1)
    assert torch.equal(out[[0, 2, 3]], got[[0, 2, 3]]) and alone.error_flags() == 0


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rot,T,Hq", [(128, 3, 4), (32, 3, 4), (64, 3000, 9)])
def test_refused_rows_of_the_paged_form_are_nan(rot, T, Hq, dtype):
    # In q's buffer and in place; rows without a sequence keep what they held.
    dev, Hkv, D = device(), 1, 128
    tab = ops.rope_table(20, rot, 1e4, dev)
    kc, vc = (torch.zeros(T, Hkv, 16, D, dtype=dtype, device=dev) for _ in range(2))
    bt = torch.arange(T, dtype=torch.int32, device=dev)[:, None].expand(T, 3).contiguous()
    lens = torch.full((T,), 5, dtype=torch.int32, device=dev)
    lens[0], lens[1] = 21, 0
    q, k, v = (torch.randn(T, h, D, generator=gen(h), device=dev).to(dtype) for h in (Hq, 1, 1))
    for qo in (torch.full_like(q, 3.0), q):
        err = torch.zeros(1, dtype=torch.int32, device=dev)
        was = qo[1].clone()
        ops.xs_qk_norm_rope_append_paged(qo, q, k, v, None, None, 1e-6, tab, kc, vc, bt, lens, err_flag=err)
        assert int(err) == ops.FLAG_BAD_LEN
        assert bool(qo[0].isnan().all()) and torch.equal(qo[1], was) and bool(qo[2:].isfinite().all())
        assert bool((kc[0] == 0).all()) and bool((vc[0] == 0).all()) and bool((vc[2, :, 4] == v[2]).all())
