"""Eviction of sequences that end on their table's last page, under tables of odd and
even widths and about the limits of the forms that rank."""
import pytest
import torch

from tests.test_gpu_evict import State

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [7, 8, 33, 255, 256, 257, 259])
@pytest.mark.parametrize("short", [0, 5, 15])
def test_to_the_tables_end(width, short):
    n = width * 16 - short
    s = State([n, 60, n - 1], 2, 2, 64, torch.bfloat16, n, width=width, draw="ties" if short == 5 else "spread")
    s.run([2, 0, 1], 3, 17, 50, 70)
