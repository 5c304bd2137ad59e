"""kda_paged_decode_q8 where the scale, or its product with a head's queries, is 0 or next to it and K's scales are large."""
import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,size", [(0.0, 1.0), (-0.0, 1.0), (2.0 ** -126, 2.0 ** 20), (2.0 ** -120, 2.0 ** -8), (-2.0 ** -149, 2.0 ** 30)])
@pytest.mark.parametrize("d,G", [(128, 4), (64, 16), (128, 24)])
def test_small_factors(d, G, scale, size, dtype):
    """Scores between 0 and a few thousandths of 2^100 2^-126: the queries' rounding, by 2^-10 of a code, moves them by
    less than 2^-15, so that the bounds of any other query hold."""
    dev = need_gpu()
    lens, ps, B, H = [300, 70, 1], 32, 16, 2
    g = torch.Generator().manual_seed(d + G)
    P = 14
    table = torch.stack([torch.nn.functional.pad(x, (0, 10 - len(x)), value=-1) for x in
                         torch.randperm(P, generator=g).to(torch.int32).split([10, 3, 1])]).contiguous()
    kc, vc = ((torch.randn(P, H, ps, d, generator=g) * 60).to(E4M3) for _ in range(2))
    vc = (vc.float().abs() + 16).to(E4M3)
    ks, vs = torch.full((P, H, ps // B), 2.0 ** 100), torch.full((P, H, ps // B), 2.0 ** -7)
    q = (torch.randn(len(lens), G * H, d, generator=g) * size).to(dtype)
    case = (q, kc, vc, ks, vs, table)
    got, lse = paged_decode_q8(*(t.to(dev) for t in case), torch.tensor(lens, dtype=torch.int32, device=dev), scale=scale,
                               return_lse=True)
    want, wl = ref.decode(*case, lens, scale)
    ref.close("out", got, want)
    layers_ref.close("lse", lse, wl)
