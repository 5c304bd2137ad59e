"""kda_paged_decode_q8 where one token's score, of up to 2^25, stands out: the output is that token's value, whatever
rounding does to the exponents of numbers of that size."""
import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3
FORMS = [(32, 3), (32, 16), (32, 20), (64, 8), (64, 11), (64, 33), (128, 8), (128, 16), (128, 24)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("bits", [17, 20, 22, 23, 24, 25])
@pytest.mark.parametrize("d,G", FORMS)
def test_one_token_stands_out(d, G, bits, apart, dtype):
    """Scores are 0 but for one token a row, whose score is between 2^(bits - 1) and 2^bits, in base 2.  Its weight is 1, the
    others' 0: for bf16 the weight's two parts (2^-8, after float16's 2^-11) and the output (2^-8) are all that is rounded,
    and what the weight is relative to, which rounds the same way in the sum.  (2^-8 + 2^-11)(1 + 2^-8) + 2^-8 < 2^-6.9.)"""
    dev = need_gpu()
    ps, B, H = 32, 16, 2
    lens = [1, 40, 130, 300, 513] * 6
    g = torch.Generator().manual_seed(d + G + bits)
    need = [-(-n // ps) for n in lens]
    P = sum(need)
    ids = torch.randperm(P, generator=g).to(torch.int32).tolist()
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    k, vc = torch.zeros(P, H, ps, d), torch.exp2(torch.randint(-3, 8, (P, H, ps, d), generator=g).float()) * 1.25
    ks = torch.full((P, H, ps // B), 1.0)
    vs = torch.exp2(torch.randint(-9, 1, ks.shape, generator=g).float()) if apart else torch.full_like(ks, 2.0 ** -4)
    for i, n in enumerate(lens):
        for j in range(need[i]):
            table[i, j] = ids.pop()
        t = int(torch.randint(0, n, (), generator=g))
        k[int(table[i, t // ps]), :, t % ps] = 16.0 + 2 * torch.randint(0, 8, (H, d), generator=g).float()
    kc, vc = k.to(E4M3), vc.to(E4M3)
    q = (1 + torch.rand(len(lens), G * H, d, generator=g)).to(dtype)
    # the largest score below 2^bits / log2 e
    most = max(float(q[i].double().abs().sum(-1).max()) for i in range(len(lens))) * 30
    scale = 2.0 ** bits * 0.6931 / most
    case = (q, kc, vc, ks, vs, table)
    got, lse = paged_decode_q8(*(t.to(dev) for t in case), torch.tensor(lens, dtype=torch.int32, device=dev), scale=scale,
                               return_lse=True)
    scale = float(torch.tensor(scale, dtype=F32))
    want, wl = ref.decode(*case, lens, scale)
    off = ((got.cpu().double() - want) / want).abs()
    assert float(off.max()) <= (2.0 ** -6.9 if dtype is BF else 2.0 ** -20), float(off.max())
    layers_ref.close("lse", lse, wl)
