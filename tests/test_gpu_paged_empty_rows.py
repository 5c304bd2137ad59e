"""Rows without tokens in every form of kda_paged_decode: zeros and -inf, whoever writes them, beside rows with some."""
import pytest
import torch

import layers_ref
from gated_delta_rule_46_gb300 import paged_decode
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,d,G,ps", [(F32, 128, 4, 16), (F32, 32, 8, 16), (BF, 128, 4, 16), (BF, 64, 32, 16), (BF, 128, 20, 64),
                                          (BF, 32, 4, 16), (BF, 64, 8, 4)])
@pytest.mark.parametrize("lens,cols", [([0], 1), ([0], 40), ([0, 0, 0], 40), ([0, 5, 0], 1), ([0, 150, 0, 0, 33, 0], 40), ([300] + [0] * 70, 80),
                                       ([0] * 70 + [61], 80), ([-3, 20, 0, -2 ** 31], 40)])
def test_empty_rows(dtype, d, G, ps, lens, cols):
    dev = need_gpu()
    if any(n > cols * ps for n in lens):
        lens = [min(n, cols * ps) for n in lens]
    g = torch.Generator().manual_seed(d + G + len(lens))
    N, H, P = len(lens), 2, sum(-(-max(n, 0) // ps) for n in lens) + 1
    kc, vc = (torch.randn(P, H, ps, d, generator=g).to(dtype) for _ in range(2))
    ids = torch.randperm(P, generator=g).to(torch.int32).tolist()
    table = torch.full((N, cols), -1, dtype=torch.int32)
    for i, n in enumerate(lens):
        for j in range(-(-max(n, 0) // ps)):
            table[i, j] = ids.pop()
    q = torch.randn(N, G * H, d, generator=g).to(dtype)
    out, lse = torch.full((N, G * H, d), float("nan"), dtype=dtype, device=dev), torch.full((N, G * H), 7.0, device=dev)
    paged_decode(q.to(dev), kc.to(dev), vc.to(dev), table.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), out=out, lse=lse)
    want, wl = layers_ref.paged(q, kc, vc, table, [max(n, 0) for n in lens], d ** -0.5)
    for i, n in enumerate(lens):
        if n <= 0:
            assert not out[i].any() and torch.isneginf(lse[i]).all()
    layers_ref.close("out", out, want)
    layers_ref.close("lse", lse, wl)
