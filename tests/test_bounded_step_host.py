"""What a bounded step refuses when it is made."""
import pytest
import torch

from paged_kv_cache_xs_gb300 import build as xsbuild
from paged_kv_cache_xs_gb300.step import BoundedDecodeStep


def test_a_limit_that_the_table_does_not_reach():
    # A sequence is cut when it is longer than the limit, and a table of 4 pages holds 64 tokens.
    xsbuild.build()

    def make(budget, **kw):
        return BoundedDecodeStep(1, 2, 2, 64, 4, 1, torch.bfloat16, "cpu", budget, **kw)

    for budget, limit in ((64, None), (10, 64), (10, 65), (1000, None), (10, 1 << 20)):
        with pytest.raises(ValueError, match="table"):
            make(budget, limit=limit)
    assert make(63).limit == 63 and make(10, limit=63).limit == 63 and make(1).limit == 1
