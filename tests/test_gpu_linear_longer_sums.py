"""Float32 outputs of linear where one CTA has all of a long K.  The tensor cores'
own sums lose up to an ulp at each step of 16 products, always towards zero, so a
sum must not run on for longer the longer K is: parts of 512 products, 512 / 16
2^-24 for one of them, and K / 512 2^-24 for adding them up in float32."""
import pytest
import torch

from gated_delta_rule_46_gb300 import linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(200, 9728, 16384), (200, 9728, 65536),   # more tiles than clusters of them fit
                                   (16, 19456, 32768), (140, 9732, 16384),
                                   (200, 9728, 32767),                       # rows that no TMA copy can start on
                                   (40, 256, 1 << 19),                       # K over a cluster, still long for each
                                   (600, 2050, 32768)])                      # no TMA store of the output
def test_parts_stay_short(M, N, K):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(K + M)
    # products of one sign: partial sums grow steadily, the worst for a loss at each step
    x = (torch.rand(M, K, generator=g, device=dev) + 0.1).to(torch.bfloat16)
    w = (torch.rand(N, K, generator=g, device=dev) + 0.1).to(torch.bfloat16)
    got = linear(x, w, out_dtype=torch.float32).double()
    want = torch.zeros(M, N, dtype=torch.float64, device=dev)
    for k in range(0, K, 8192):
        want += x[:, k:k + 8192].double() @ w[:, k:k + 8192].double().t()
    err = ((got - want).norm() / want.norm()).item()
    tol = (512 / 16 + K / 512) * 2.0 ** -24
    assert err <= tol, f"{err:.2e} > {tol:.2e}"
