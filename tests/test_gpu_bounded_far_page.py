"""Decode attention where one page's logits lie so far below all others that its
weights are exactly 0: the outputs are those of the other pages."""
import pytest
import torch

from tests import plain_bounded as plain
from tests.gpu_helpers import device
from tests.test_gpu_bounded_decode import BF, F32, Case, near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("far", [0, 3])
@pytest.mark.parametrize("B", [1, 40, 90], ids=["cluster", "ctas", "line"])
def test_a_page_far_below_the_others(B, far, dtype):
    n = 100
    c = Case([n] * B, 8, 2, 128, dtype, 12, width=150 if B == 90 else None)
    # Queries below 0 on keys above it, those of one page 1e30 times as large: logits of -1e30 and less.
    c.q.copy_(-c.q.abs()), c.k.abs_()
    for b in range(B):
        c.k[int(c.tables[b, far])] *= 1e30
    c.d["q"].copy_(c.q), c.d["k"].copy_(c.k)
    ws = c.workspace(True)
    scores = torch.zeros(B, 2, c.tables.shape[1] * 16, device=device())
    at = [t for t in range(n) if t // 16 != far]
    want = [plain.attend(c.q[b], plain.rows(c.k, c.tables[b].tolist(), at), plain.rows(c.v, c.tables[b].tolist(), at), c.scale)
            for b in range(B)]
    ref = torch.stack([w[0] for w in want])
    bound = torch.stack([plain.out_bound(w[0], w[2], w[3], dtype, 15 if dtype == BF else 20) for w in want])
    near(c.first_call(ws), ref, bound, "first")
    near(c.weights_call(ws, scores), ref, bound, "weights")
    for b in range(B):
        _, p, _, slack = want[b]
        add = p.view(2, 4, -1).sum(1)
        off = (p * (2 * slack[:, None] + 2.0 ** -20)).view(2, 4, -1).sum(1) + 6 * 2.0 ** -24 * add + 1e-30
        near(scores[b][:, at], add, off, f"scores of {b}")
        assert int(scores[b, :, 16 * far:16 * far + 16].count_nonzero()) == 0
    assert int(c.err) == 0
