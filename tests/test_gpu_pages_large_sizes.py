"""Sizes that 32 bits do not hold are refused by the pages' bindings, not cut short."""
import pytest
import torch

from gated_delta_rule_46_gb300 import pages_compact, pages_fork, pages_resize
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page_size", [(1 << 32) + 16, -(1 << 32) + 16, -16])
def test_page_size(page_size):
    dev = need_gpu()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    with pytest.raises(ValueError):
        pages_resize(i(3, 4), i(3), i(9), i(3), page_size)
    with pytest.raises(ValueError):
        pages_fork([], i(3, 4), i(3), i(9), i(3), i(1), i(1), page_size)


def test_tables_and_counts():
    """(Neither is written or read: a refused call does nothing.)"""
    dev = need_gpu()
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)  # noqa: E731
    n = (1 << 32) + 9
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB of device memory")
    long = torch.empty(n, dtype=torch.int32, device=dev)
    with pytest.raises(ValueError):
        pages_resize(i(3, 4), i(3), long, i(3), 16)
    with pytest.raises(ValueError):
        pages_resize(long[None], i(1), i(9), i(1), 16)
    with pytest.raises(ValueError):
        pages_fork([], long[None], i(1), i(9), i(1), i(1), i(1), 16)
    with pytest.raises(ValueError):
        pages_compact([], None, long)
    with pytest.raises(ValueError):
        pages_compact([], long[None], i(9))
