"""kda_paged_decode_q8 over values as small as kda_paged_append_q8 stores them: scales down to 2^-126."""
import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import paged_append_q8, paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3
FORMS = [(32, 3), (32, 16), (32, 20), (64, 8), (64, 11), (64, 33), (128, 8), (128, 16), (128, 24)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("e", [-126, -118, -109, -101, -90])
@pytest.mark.parametrize("d,G", FORMS)
def test_scales_next_to_the_smallest(d, G, e, dtype):
    """All scales of V the same: the outputs are the power of two times those of scales of 1, whose codes are 8 to 384 in
    size and whose weights are not far apart, so that no product of a weight and a value comes below 2^-130, where float32
    keeps multiples of 2^-149: off by 2^-20 of it."""
    dev = need_gpu()
    lens, ps, B, H = [90, 300, 1], 32, 16, 2
    g = torch.Generator().manual_seed(d + G)
    P = 14
    table = torch.randperm(P, generator=g)[:P].to(torch.int32)
    table = torch.stack([torch.nn.functional.pad(x, (0, 10 - len(x)), value=-1) for x in table.split([3, 10, 1])]).contiguous()
    kc = (torch.randn(P, H, ps, d, generator=g) / 8).to(E4M3)
    vc = (torch.exp2(torch.randint(3, 9, (P, H, ps, d), generator=g).float()) * torch.where(torch.rand(P, H, ps, d, generator=g) < 0.5, 1.0, 1.5)).to(E4M3)
    ks, vs = torch.ones(P, H, ps // B), torch.full((P, H, ps // B), 2.0 ** e)
    q = torch.randn(len(lens), G * H, d, generator=g).to(dtype)
    case = (q, kc, vc, ks, vs, table)
    got, lse = paged_decode_q8(*(t.to(dev) for t in case), torch.tensor(lens, dtype=torch.int32, device=dev), return_lse=True)
    want, wl = ref.decode(*case, lens, d ** -0.5)
    layers_ref.close("lse", lse, wl)
    e_rel, most = layers_ref.rel(got.double() * 2.0 ** 90, want * 2.0 ** 90), ref.BF16_TOL if dtype is BF else ref.F32_TOL
    assert e_rel <= most, f"rel-L2 {e_rel:.3e} > {most:.3e}"


@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_values_appended_and_read(dtype):
    """Values of 2^-118 and less through both calls."""
    dev = need_gpu()
    n, H, d, ps, B = 70, 2, 64, 32, 16
    g = torch.Generator().manual_seed(3)
    k, v = torch.randn(n, H, d, generator=g), torch.randn(n, H, d, generator=g).clamp(-4, 4) * 2.0 ** -119
    kc, vc = (torch.zeros(4, H, ps, d, dtype=torch.uint8, device=dev).view(E4M3) for _ in range(2))
    ks, vs = (torch.zeros(4, H, ps // B, device=dev) for _ in range(2))
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    paged_append_q8(k.to(dtype).to(dev), v.to(dtype).to(dev), kc, vc, ks, vs, table, i32([0]), cu_seqlens=i32([0, n]))
    q = torch.randn(1, 4 * H, d, generator=g).to(dtype)
    got = paged_decode_q8(q.to(dev), kc, vc, ks, vs, table, i32([n]))
    want, _ = ref.decode(q, *(t.cpu() for t in (kc, vc, ks, vs, table)), [n], d ** -0.5)
    e, most = layers_ref.rel(got.double() * 2.0 ** 119, want * 2.0 ** 119), ref.BF16_TOL if dtype is BF else ref.F32_TOL
    assert e <= most, f"rel-L2 {e:.3e} > {most:.3e}"
