"""Decays that leave nothing of the past: lambda is 0 in float32, lambda^0 is 1.
With q and k the same unit vector the output is then v itself, which bf16 and
float32 hold exactly: every weight but the diagonal's is 0, and that one is 1."""
import math

import pytest
import torch

from gated_delta_rule_46_gb300 import decay_decode, decay_prefill
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
RATES = [-200.0, -1000.0, -3000.0, -5000.0, -9000.0, -11000.0, -20000.0, -math.inf]


def _unit(T, H, d, dtype, dev):
    x = torch.zeros(T, H, d, dtype=dtype, device=dev)
    x[..., 5] = 1
    return x


@pytest.mark.parametrize("dtype,dk,dv", [(BF, 128, 128), (BF, 64, 64), (BF, 32, 32), (BF, 64, 128), (F32, 128, 128), (F32, 32, 64)])
@pytest.mark.parametrize("lens", [[300, 1, 64], [2500], [40] * 50])
def test_output_is_the_token_s_own_value(dtype, dk, dv, lens):
    dev = need_gpu()
    T, H = sum(lens), len(RATES)
    q = _unit(T, H, dk, dtype, dev)
    v = torch.randn(T, H, dv, generator=torch.Generator().manual_seed(dk + T)).to(dtype).to(dev)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    init = torch.randn(len(lens), H, dk, dv, generator=torch.Generator().manual_seed(1)).to(dev)
    out, fin = decay_prefill(q, q, v, torch.tensor(RATES, device=dev), cu, init)
    bad = [r for i, r in enumerate(RATES) if not torch.equal(out[:, i], v[:, i])]
    assert not bad, f"log-decays {bad}"
    want = torch.zeros_like(fin)
    want[:, :, 5] = v[cu[1:].long() - 1].float()
    assert torch.equal(fin, want)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("lens", [[130, 0, 5], [2500], [40] * 50])
def test_a_nan_decay_is_not_taken_for_a_number(dtype, d, lens):
    """exp(NaN) S is NaN from the first token on; the other heads and the sequences without tokens are as before."""
    dev = need_gpu()
    T, g = sum(lens), torch.Generator().manual_seed(7)
    q, k, v = (torch.randn(T, 3, d, generator=g).to(dtype).to(dev) / d ** 0.25 for _ in range(3))
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    init = torch.randn(len(lens), 3, d, d, generator=g).to(dev)
    rates = torch.tensor([-0.5, -0.25, -1.0], device=dev)
    clean, cfin = decay_prefill(q, k, v, rates, cu, init)
    rates[1] = math.nan
    out, fin = decay_prefill(q, k, v, rates, cu, init)
    assert torch.isnan(out[:, 1]).all()
    assert torch.equal(out[:, ::2], clean[:, ::2]) and torch.equal(fin[:, ::2], cfin[:, ::2])
    for i, n in enumerate(lens):
        assert torch.isnan(fin[i, 1]).all() if n else torch.equal(fin[i, 1], init[i, 1])


def test_decode_agrees():
    dev = need_gpu()
    H, d = len(RATES) + 1, 64
    q = _unit(2, H, d, F32, dev)
    v = torch.randn(2, H, d, generator=torch.Generator().manual_seed(3)).to(dev)
    pool = torch.randn(2, H, d, d, generator=torch.Generator().manual_seed(4)).to(dev)
    out = decay_decode(q, q, v, torch.tensor(RATES + [math.nan], device=dev), pool)
    assert torch.equal(out[:, :-1], v[:, :-1]) and torch.isnan(out[:, -1]).all()
