"""kda_paged_decode_q8 over a cache of more than 2^31 rows, and over none."""
import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import check_device_status, kda, paged_append_q8, paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("d,H,ps,B,G", [(32, 8, 128, 128, 4), (32, 2, 1024, 128, 17)])
def test_rows_past_31_bits(d, H, ps, B, G):
    """Pages at both ends of the cache and on either side of row 2^31, appended to and read (keys and values are one tensor)."""
    dev = need_gpu()
    P = (1 << 31) // (H * ps) + 40
    if torch.cuda.mem_get_info()[0] < P * H * ps * d + (4 << 30):
        pytest.skip("needs 70 GB of device memory")
    cache = torch.empty(P, H, ps, d, dtype=torch.uint8, device=dev).view(E4M3)
    scales = torch.zeros(P, H, ps // B, device=dev)
    mid = (1 << 31) // (H * ps)
    rows = [[P - 1, 0, mid, mid - 1], [mid + 7, P - 2, 1, -1], [mid + 1, 2, -1, -1]]
    lens = [3 * ps + 77, 2 * ps + 5, ps + 1]
    g = torch.Generator().manual_seed(d + H)
    k = torch.randn(sum(lens), H, d, generator=g)
    table = _i32(rows, dev)
    kd = k.to(dev)
    paged_append_q8(kd, kd, cache, cache, scales, scales, table, _i32([0] * 3, dev),
                    cu_seqlens=_i32([0] + torch.tensor(lens).cumsum(0).tolist(), dev))
    # the pages in use, as a small cache
    used = sorted({p for r in rows for p in r if p >= 0})
    kc, ks = cache.view(torch.uint8)[used].cpu().view(E4M3), scales[used].cpu()
    small = torch.tensor([[used.index(p) if p >= 0 else -1 for p in r] for r in rows], dtype=torch.int32)
    code, want = torch.zeros(kc.shape, dtype=torch.float64), torch.zeros(ks.shape, dtype=torch.float64)
    ref.append(k, code, want, small, [0] * 3, lens)
    ref.same("scales", ks, want)
    for i, n in enumerate(lens):
        for j in range(-(-n // ps)):
            m = min(ps, n - j * ps)
            ref.same("codes", kc[small[i, j], :, :m], code[small[i, j], :, :m])
    for dtype in (BF, F32):
        q = torch.randn(3, G * H, d, generator=g).to(dtype)
        status = torch.zeros(4, dtype=torch.int32, device=dev)
        out, lse = paged_decode_q8(q.to(dev), cache, cache, scales, scales, table, _i32(lens, dev), return_lse=True, status=status)
        assert check_device_status(status) == kda.KDA_OK
        wo, wl = ref.decode(q, kc, kc, ks, ks, small, lens, d ** -0.5)
        ref.close("out", out, wo)
        layers_ref.close("lse", lse, wl)
    del cache
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pages,cols", [(0, 3), (0, 0), (3, 0)])
@pytest.mark.parametrize("N,d,G", [(3, 64, 4), (5000, 32, 1), (40, 128, 20)])
def test_no_pages(N, d, G, pages, cols, dtype):
    """Zeros and -inf; a length that is not 0 is recorded."""
    dev = need_gpu()
    H, ps = 2, 32
    q = torch.randn(N, G * H, d, device=dev).to(dtype)
    kc, ks = torch.zeros(pages, H, ps, d, dtype=torch.uint8, device=dev).view(E4M3), torch.ones(pages, H, 1, device=dev)
    table = torch.zeros(N, cols, dtype=torch.int32, device=dev)
    for n, want in ((0, kda.KDA_OK), (1, kda.KDA_ERR_INVALID_ARG), (-1, kda.KDA_ERR_INVALID_ARG)):
        lens = torch.zeros(N, dtype=torch.int32, device=dev)
        lens[N // 2] = n
        out, lse = torch.full((N, G * H, d), 3.0, dtype=dtype, device=dev), torch.full((N, G * H), 3.0, device=dev)
        status = torch.zeros(4, dtype=torch.int32, device=dev)
        paged_decode_q8(q, kc, kc, ks, ks, table, lens, out=out, lse=lse, status=status)
        assert check_device_status(status) == want
        assert not out.any() and torch.isneginf(lse).all()
