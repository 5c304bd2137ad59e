"""kda_linear with more rows than one launch takes (its row tiles are a grid dimension)."""
import pytest
import torch

from gated_delta_rule_46_gb300 import linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N", [5, 8])                # by rows; a float32 output that TMA can store
@pytest.mark.parametrize("K,ld", [(8, 8), (7, 9)])
def test_rows_past_a_slice(N, K, ld):
    dev = need_gpu()
    M = 4194048 + 333
    g = torch.Generator(device=dev).manual_seed(N)
    x = torch.randint(-3, 4, (M, ld), generator=g, device=dev).to(torch.bfloat16)[:, :K]
    w = torch.randint(-3, 4, (N, K), generator=g, device=dev).to(torch.bfloat16)
    r = torch.randint(-9, 10, (M, N), generator=g, device=dev).float()
    want = (x.float()[:, None, :] * w.float()).sum(2) + r          # small whole numbers: exact
    assert torch.equal(linear(x, w, residual=r, out_dtype=torch.float32), want)
