"""Prompt chunks with first tokens and a window: values near the end of bf16,
against 64 bits."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from tests import plain_bounded as plain
from tests.gpu_helpers import device
from tests.test_gpu_bounded_prefill import chunk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.mark.parametrize("T,start,Hq,Hkv", [(640, 1000, 64, 8), (16, 6000, 8, 2)], ids=["pairs", "cluster"])
def test_weights_above_the_first_tiles_do_not_overflow(T, start, Hq, Hkv):
    """Logits that rise by 6.9 powers of two behind a row's first key tile, over values
    from 2^120 on: a weight above 1 would make infinities of them."""
    g = torch.Generator().manual_seed(start)
    q, k, v, ids = chunk(T, start, Hq, Hkv, 64, 3, 0, 0)
    q.fill_(1.0)
    n = start + T
    at = torch.arange(-(-n // 16) * 16)
    logit = torch.zeros(at.numel())
    logit[(at < n) & ((at // 128 % 5 == 2) | (at // 128 % 5 == 3)) & (at % 128 < 2)] = 4.75
    k[ids.long()[at // 16], :, at % 16] = (logit / 64).to(BF)[:, None, None].expand(-1, Hkv, 64)
    v.copy_(((0.5 + torch.rand(v.shape, generator=g)) * 2.0 ** 121).to(BF))
    out, err = torch.full(q.shape, 7.0, dtype=BF, device=device()), torch.zeros(1, dtype=torch.int32, device=device())
    ops.xs_paged_prefill_first(out, *(x.to(device()) for x in (q, k, v, ids)), start, 1.0, err_flag=err)
    out = out.cpu().double()
    assert int(err) == 0 and bool(out.isfinite().all())
    for i in (0, T // 2, T - 1):
        seen = plain.seen_by(start + i + 1, 0, 0)
        ref, _, mag, slack = plain.attend(q[i], plain.rows(k, ids.tolist(), seen), plain.rows(v, ids.tolist(), seen), 1.0)
        d = (out[i] - ref).abs()
        assert bool((d <= plain.out_bound(ref, mag, slack, BF, 8)).all()), i
