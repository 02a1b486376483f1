"""Sequences cut into pages that they share with others."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import ops
from paged_kv_cache_xs_gb300.step import BoundedDecodeStep
from tests.gpu_helpers import device
from tests.test_gpu_share import Both, i32

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def append(s, k, v, rows):
    """One token to every sequence; rows [B, Hkv, D]."""
    ops.xs_block_alloc_decode(s.tables, s.lens, s.stack, s.top)
    slots = torch.empty(s.lens.numel(), dtype=torch.int64, device=device())
    ops.xs_slot_mapping(s.tables, s.lens, 16, k.shape[0], slots)
    ops.xs_kv_append(rows, rows, k, v, slots)


def text(s, k, b):
    """The rows of sequence b's tokens."""
    n = int(s.lens[b])
    at = torch.arange(n, device=device())
    return k[s.tables[b, at // 16].long(), :, at % 16]


def test_an_append_behind_a_cut_into_a_shared_page():
    """As documented: fork into an empty slot, copy, release; the other owner keeps its rows."""
    s = Both([100, -1, -1], 8, 30, seed=1)
    g = torch.Generator(device=device()).manual_seed(1)
    k, v = (torch.randn(30, 2, 16, 64, generator=g, device=device()).to(BF) for _ in range(2))
    whole = text(s, k, 0).clone()
    ops.xs_block_copy(k[None], v[None], s.fork([0], [1]))
    ops.xs_block_truncate(i32([1]), i32([40]), s.tables, s.lens, s.stack, s.top, s.extra, err_flag=s.err)
    copies = torch.zeros(1, 2, dtype=torch.int64, device=device())
    ops.xs_block_fork(i32([1]), i32([2]), s.tables, s.lens, s.stack, s.top, s.extra, copies, err_flag=s.err)
    ops.xs_block_copy(k[None], v[None], copies)
    ops.xs_block_release(i32([1]), s.tables, s.lens, s.stack, s.top, s.extra, err_flag=s.err)
    assert s.lens.tolist() == [100, -1, 40] and int(s.err) == 0
    for t in range(20):
        rows = torch.randn(3, 2, 64, generator=g, device=device()).to(BF)
        append(s, k, v, rows)
        assert torch.equal(text(s, k, 2)[40 + t], rows[2]) and torch.equal(text(s, k, 0)[100 + t], rows[0])
    assert torch.equal(text(s, k, 0)[:100], whole) and torch.equal(text(s, k, 2)[:40], whole[:40])
    used = [i for b in (0, 2) for i in s.tables[b].tolist() if i >= 0]
    assert s.extra.tolist() == [max(0, used.count(i) - 1) for i in range(30)]
    assert sorted(s.stack.tolist()[:int(s.top)]) == [i for i in range(30) if i not in used]


def test_a_step_that_keeps_the_first_tokens_alone():
    """Two sequences share the page in which the budget ends: they are not cut, as one that
    shares a page which the eviction writes; a third one is."""
    s = Both([32, -1, 33], 6, 20, seed=2)
    s.fork([0], [1])
    step = BoundedDecodeStep(3, 4, 2, 64, 6, 1, BF, device(), budget=20, limit=30, first=20)
    g = torch.Generator(device=device()).manual_seed(2)
    k, v = (torch.randn(1, 20, 2, 16, 64, generator=g, device=device()).to(BF) for _ in range(2))
    before = [text(s, k[0], b).clone() for b in range(3)]
    step.bound(k, v, s.tables, s.lens, s.stack, s.top, s.extra)
    assert s.lens.tolist() == [32, 32, 20] and step.error_flags() == ops.FLAG_SHARED
    assert step.new_lens.tolist() == [-1, -1, 20] and step.scored.tolist() == [32, 32, 20]
    assert step.kept[0, :, 0].tolist() == [[-1] * 20] * 2 + [list(range(20))]
    append(s, k[0], v[0], torch.randn(3, 2, 64, generator=g, device=device()).to(BF))
    for b in range(3):
        assert torch.equal(text(s, k[0], b)[:-1], before[b][:int(s.lens[b]) - 1])
    # With the other released, it is cut.
    ops.xs_block_release(i32([0]), s.tables, s.lens, s.stack, s.top, s.extra)
    step.bound(k, v, s.tables, s.lens, s.stack, s.top, s.extra)
    assert s.lens.tolist() == [-1, 20, 21]
