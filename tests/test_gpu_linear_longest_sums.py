"""bf16 outputs of linear at K far past a model's widths.  The tensor cores' own sums
lose up to an ulp, 2^-23 of themselves, at each step of 16 products, always towards
zero: in parts of at most 65536 products that is 2^-11 of the result, where its
rounding to bf16 takes 2^-9.  No wait in a kernel lasts for more than one such part."""
import pytest
import torch

from gated_delta_rule_46_gb300 import check_device_status, kda, linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(600, 2048, 1 << 20),      # as many rows as pairs of CTAs take
                                   (4, 64, 1 << 24),          # K over a cluster
                                   (4, 64, (1 << 22) + 1),    # rows that no TMA copy can start on
                                   (1, 1, 1 << 30),
                                   (1, 1, (1 << 30) + 1)])    # seconds of work for one cluster
def test_bf16_output_at_very_long_k(M, N, K):
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(M + N)

    def rand(n):
        t = torch.empty(n, K, dtype=torch.bfloat16, device=dev)
        for k in range(0, K, 1 << 24):
            t[:, k:k + (1 << 24)] = torch.rand(n, min(K - k, 1 << 24), generator=g, device=dev) + 0.1
        return t
    x, w = rand(M), rand(N)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = linear(x, w, status=status).double()
    assert check_device_status(status) == kda.KDA_OK
    step = max(1, (1 << 26) // max(M, N))
    want = torch.zeros(M, N, dtype=torch.float64, device=dev)
    for k in range(0, K, step):
        want += x[:, k:k + step].double() @ w[:, k:k + step].double().t()
    err = ((got - want).norm() / want.norm()).item()
    assert err <= 2.0 ** -9 + 2.0 ** -11, f"{err:.2e}"
