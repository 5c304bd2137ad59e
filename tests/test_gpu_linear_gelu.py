"""The lower tail of GELU, y Phi(y), element by element.  Taken from erfc or from
e^{-x^2} and Mills' ratio, x = y / sqrt 2, it keeps its relative precision where 1 +
erf cancels: a few ulp for the function, and the rounding of its argument (2^-24 of
it, twice) moves it by at most about 2 x^2 + 2 times that.  With x^2 <= 50 that is
below 300 2^-24."""
import pytest
import torch

from gated_delta_rule_46_gb300 import linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N", [(16, 40), (64, 256), (2600, 520)])      # split over K or not; pairs of CTAs
def test_lower_tail(M, N):
    dev = need_gpu()
    y = torch.linspace(-10, 4, M * N, dtype=torch.float64).to(torch.bfloat16).reshape(M, N)
    w = torch.eye(N, dtype=torch.bfloat16)
    want = 0.5 * y.double() * torch.special.erfc(-y.double() / 2 ** 0.5)
    got = linear(y.to(dev), w.to(dev), act="gelu", out_dtype=torch.float32).cpu().double()
    assert float(((got - want).abs() / want.abs().clamp(min=1e-300)).max()) <= 300 * 2.0 ** -24
    got = linear(y.to(dev), w.to(dev), act="gelu").cpu().double()
    assert float(((got - want).abs() / want.abs().clamp(min=1e-300)).max()) <= 300 * 2.0 ** -24 + 2.0 ** -8
