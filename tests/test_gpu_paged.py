"""The paged key-value cache (kda_paged_append) and attention over it
(kda_paged_decode) against float64."""
import math

import pytest
import torch

import layers_ref as ref
from gated_delta_rule_46_gb300 import (KDAError, check_device_status, kda, paged_append, paged_decode,
                                       paged_decode_workspace_size)
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _cache(lens, Hkv, G, d, ps, dtype, seed, extra_cols=1):
    """Random pages, what no token was written to NaN; table entries past a sequence's pages are -1."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    P, cols = sum(need) + 2, max(need + [0]) + extra_cols
    kc = torch.full((P, Hkv, ps, d), math.nan, dtype=dtype)
    vc = kc.clone()
    table = torch.full((len(lens), cols), -1, dtype=torch.int32)
    ids = torch.randperm(P, generator=g).tolist()
    for i, n in enumerate(lens):
        for j in range(need[i]):
            p = ids.pop()
            table[i, j] = p
            m = min(ps, n - j * ps)
            kc[p, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
            vc[p, :, :m] = torch.randn(Hkv, m, d, generator=g).to(dtype)
    q = torch.randn(len(lens), Hkv * G, d, generator=g).to(dtype)
    return q, kc, vc, table


def _decode(q, kc, vc, table, lens, dev, **kw):
    return paged_decode(q.to(dev), kc.to(dev), vc.to(dev), table.to(dev),
                        torch.tensor(lens, dtype=torch.int32, device=dev), return_lse=True, **kw)


def _check(q, kc, vc, table, lens, dev, scale=None, **kw):
    out, lse = _decode(q, kc, vc, table, lens, dev, scale=scale, **kw)
    ro, rl = ref.paged(q, kc, vc, table, lens, q.shape[2] ** -0.5 if scale is None else scale)
    ref.close("out", out, ro)
    ref.close("lse", lse, rl)
    return out, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ps", [1, 4, 8, 16, 64, 128, 256, 1024])
def test_page_sizes(dtype, d, ps):
    dev = need_gpu()
    lens = [1, ps, ps + 1, 0, 130, 300]
    _check(*_cache(lens, 2, 3, d, ps, dtype, seed=ps + d), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hkv,G", [(1, 1), (3, 1), (1, 2), (2, 5), (1, 8), (2, 12), (1, 16), (1, 17), (2, 33), (1, 64)])
def test_head_layouts(dtype, Hkv, G):
    dev = need_gpu()
    lens = [77, 1, 200]
    _check(*_cache(lens, Hkv, G, 128, 32, dtype, seed=G), lens, dev, scale=0.3)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 385])
def test_lengths(dtype, d, n):
    """Lengths that end inside a page and inside a tile."""
    dev = need_gpu()
    _check(*_cache([n, 0, n + 1], 2, 4, d, 16, dtype, seed=n), [n, 0, n + 1], dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens", [[5000], [0, 0, 7000, 0], [3, 4000, 1, 2900], [0], [0, 0]])
def test_long_rows_split_and_joined(dtype, lens):
    dev = need_gpu()
    _check(*_cache(lens, 2, 4, 128, 64, dtype, seed=len(lens)), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_sequences(dtype):
    """More (sequence, head) items than the grid has blocks, and more sequences than threads in one."""
    dev = need_gpu()
    g = torch.Generator().manual_seed(1)
    lens = [int(x) for x in torch.randint(0, 40, (700,), generator=g)]
    _check(*_cache(lens, 2, 2, 64, 16, dtype, seed=2), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sharp_and_large_scores(dtype):
    """Scores of some hundreds: the softmax picks one token; the running maximum moves late in the row."""
    dev = need_gpu()
    lens = [1500, 90]
    q, kc, vc, table = _cache(lens, 1, 4, 128, 64, dtype, seed=3)
    kc[int(table[0, 1400 // 64]), 0, 1400 % 64] = 8 * q[0, 2]
    _check(q, kc, vc, table, lens, dev, scale=1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_unused_slots_and_neighbours_do_not_leak(dtype):
    """The cache holds NaN wherever no token was written (so in every case above); here infinities as
    well, and one sequence whose own token is NaN."""
    dev = need_gpu()
    lens = [70, 100, 129]
    q, kc, vc, table = _cache(lens, 2, 4, 128, 32, dtype, seed=4)
    kc[torch.isnan(kc)] = math.inf
    vc[torch.isnan(vc)] = -math.inf
    _check(q, kc, vc, table, lens, dev)
    vc[int(table[1, 0]), 1, 5, 7] = math.nan
    out, lse = _decode(q, kc, vc, table, lens, dev)
    bad = torch.isnan(out).cpu()
    assert bad[1, 4:, 7].all() and int(bad.sum()) == 4 and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_pages_and_lengths_are_reported_and_left_out(dtype):
    dev = need_gpu()
    lens = [200, 64, 100, 40]
    q, kc, vc, table = _cache(lens, 2, 4, 128, 32, dtype, seed=5, extra_cols=0)
    table[0, 2] = kc.shape[0]                                      # tokens 64..95 on a page outside the cache
    table[1, :2] = -7                                              # nothing left
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    ro, rl = ref.paged(q, kc, vc, table, lens, 128 ** -0.5)
    out, lse = _decode(q, kc, vc, table, lens, dev, status=status)
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    ref.close("out", out, ro)
    ref.close("lse", lse, rl)
    assert torch.count_nonzero(out[1]) == 0 and (lse[1] == -math.inf).all()
    # a negative length is 0, one past the table is the table's end
    q, kc, vc, table = _cache([224, 10], 2, 4, 128, 32, dtype, seed=6, extra_cols=0)
    for bad, real in (([224, -5], [224, 0]), ([225, 10], [224, 10]), ([2 ** 31 - 1, 10], [224, 10])):
        status.zero_()
        out, lse = _decode(q, kc, vc, table, bad, dev, status=status)
        assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
        ro, rl = ref.paged(q, kc, vc, table, real, 128 ** -0.5)
        ref.close("out", out, ro)
        ref.close("lse", lse, rl)
    status.zero_()
    _decode(q, kc, vc, table, [224, 10], dev, status=status)
    assert check_device_status(status) == kda.KDA_OK


def test_row_stride_workspace_stream_and_repeats():
    dev = need_gpu()
    lens = [900, 40, 0, 300]
    q, kc, vc, table = _cache(lens, 2, 4, 128, 64, BF, seed=7)
    out, lse = _check(q, kc, vc, table, lens, dev)
    qs, = ref.fused_rows([q], dev)
    c = [t.to(dev) for t in (kc, vc, table)]
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = torch.full((paged_decode_workspace_size(4, table.shape[1] * 64, 8, 2, 128),), 255, dtype=torch.uint8, device=dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, l2 = paged_decode(qs, *c, n, return_lse=True, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert torch.equal(out, paged_decode(qs, *c, n))


def test_offsets_past_32_bits():
    """A cache of over 2^31 elements; the pages in use lie at its end."""
    dev = need_gpu()
    ps, Hkv, d = 64, 2, 128
    P = 2 ** 31 // (ps * Hkv * d) + 40
    lens = [300, 70]
    q, kc, vc, table = _cache(lens, Hkv, 4, d, ps, BF, seed=8)
    big = [torch.zeros(P, Hkv, ps, d, dtype=BF, device=dev) for _ in range(2)]
    off = P - kc.shape[0]
    for b, c in zip(big, (kc, vc)):
        b[off:] = c.to(dev)
    t2 = torch.where(table >= 0, table + off, table)
    out, lse = paged_decode(q.to(dev), *big, t2.to(dev), torch.tensor(lens, dtype=torch.int32, device=dev), return_lse=True)
    ro, rl = ref.paged(q, kc, vc, table, lens, d ** -0.5)
    ref.close("out", out, ro)
    ref.close("lse", lse, rl)
    k = torch.randn(2, Hkv, d).to(BF).to(dev)
    paged_append(k, -k, *big, t2.to(dev), torch.tensor([299, 69], dtype=torch.int32, device=dev))
    for i, n in enumerate(lens):
        p, o = int(t2[i, (n - 1) // ps]), (n - 1) % ps
        assert torch.equal(big[0][p, :, o], k[i]) and torch.equal(big[1][p, :, o], -k[i])


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 32), (F32, 64)])
@pytest.mark.parametrize("ps", [1, 16, 128])
@pytest.mark.parametrize("fused", [False, True])
def test_append_prompts_then_tokens(dtype, d, ps, fused):
    dev = need_gpu()
    lens, starts, H = [5, 0, 130, 1, 33], [0, 7, 9, 40, 16], 3
    ends = [a + b for a, b in zip(lens, starts)]
    _, kc, vc, table = _cache([e + 1 for e in ends], H, 1, d, ps, dtype, seed=9)
    wk, wv = kc.clone(), vc.clone()
    g = torch.Generator().manual_seed(10)
    dk, dv, dt = kc.to(dev), vc.to(dev), table.to(dev)
    for L, S in ((lens, starts), ([1] * 5, ends)):
        T = sum(L)
        k, v = torch.randn(T, H, d, generator=g).to(dtype), torch.randn(T, H, d, generator=g).to(dtype)
        t = 0
        for i in range(5):
            for p in range(S[i], S[i] + L[i]):
                wk[table[i, p // ps], :, p % ps], wv[table[i, p // ps], :, p % ps] = k[t], v[t]
                t += 1
        kd, vd = ref.fused_rows([k, v], dev) if fused else (k.to(dev), v.to(dev))
        cu = None if L == [1] * 5 else torch.tensor([0] + torch.tensor(L).cumsum(0).tolist(), dtype=torch.int32, device=dev)
        paged_append(kd, vd, dk, dv, dt, torch.tensor(S, dtype=torch.int32, device=dev), cu)
    bits = lambda t: t.cpu().view(torch.int16 if dtype == BF else torch.int32)  # noqa: E731
    assert torch.equal(bits(dk), bits(wk)) and torch.equal(bits(dv), bits(wv))


def test_append_unaligned_rows():
    """Rows that start off a 16-byte boundary take the element-wise copy."""
    dev = need_gpu()
    _, kc, vc, table = _cache([20], 2, 1, 64, 16, BF, seed=11)
    flat = torch.randn(20, 2 * 2 * 64 + 3).to(BF).to(dev)
    k, v = flat[:, 1:129].unflatten(1, (2, 64)), flat[:, 129:257].unflatten(1, (2, 64))
    dk, dv = kc.to(dev), vc.to(dev)
    paged_append(k, v, dk, dv, table.to(dev), torch.zeros(1, dtype=torch.int32, device=dev),
                 torch.tensor([0, 20], dtype=torch.int32, device=dev))
    for t in range(20):
        p = int(table[0, t // 16])
        assert torch.equal(dk[p, :, t % 16], k[t]) and torch.equal(dv[p, :, t % 16], v[t])


def test_append_reports_what_has_no_place():
    dev = need_gpu()
    _, kc, vc, table = _cache([20, 20, 20], 2, 1, 64, 16, F32, seed=12, extra_cols=0)
    table[1, 1] = kc.shape[0] + 5
    dk, dv = kc.to(dev), vc.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    k = torch.randn(3, 2, 64, device=dev)
    # off the table's end, a page outside the cache, a negative position
    paged_append(k, k, dk, dv, table.to(dev), torch.tensor([32, 17, -1], dtype=torch.int32, device=dev), status=status)
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    assert torch.equal(dk.cpu().view(torch.int32), kc.view(torch.int32))
    assert torch.equal(dv.cpu().view(torch.int32), vc.view(torch.int32))


def test_append_then_attend_token_by_token():
    """A serving loop: append the new token, attend over everything so far; each step is one row of
    causal attention."""
    dev = need_gpu()
    n, Hkv, G, d, ps = 40, 2, 4, 64, 16
    g = torch.Generator().manual_seed(13)
    k, v, q = (torch.randn(n, h, d, generator=g).to(BF) for h in (Hkv, Hkv, Hkv * G))
    kc = torch.full((4, Hkv, ps, d), math.nan, dtype=BF, device=dev)
    vc = kc.clone()
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=dev)
    for t in range(n):
        paged_append(k[t:t + 1].to(dev), v[t:t + 1].to(dev), kc, vc, table, torch.tensor([t], dtype=torch.int32, device=dev))
        out = paged_decode(q[t:t + 1].to(dev), kc, vc, table, torch.tensor([t + 1], dtype=torch.int32, device=dev))
        s = torch.einsum("hgd,thd->hgt", q[t].double().reshape(Hkv, G, d), k[:t + 1].double()) * d ** -0.5
        ro = torch.einsum("hgt,thd->hgd", torch.softmax(s, -1), v[:t + 1].double()).reshape(1, Hkv * G, d)
        ref.close(f"token {t}", out, ro)


def test_refusals():
    dev = need_gpu()
    q, kc, vc, table = (t.to(dev) for t in _cache([20], 2, 2, 64, 16, BF, seed=14))
    n = torch.tensor([20], dtype=torch.int32, device=dev)
    with pytest.raises(TypeError):
        paged_decode(q.float(), kc, vc, table, n)
    with pytest.raises(ValueError):
        paged_decode(q, kc, vc[:1], table, n)
    with pytest.raises(ValueError):
        paged_decode(q, kc.transpose(1, 2), vc.transpose(1, 2), table, n)
    with pytest.raises(TypeError):
        paged_decode(q, kc, vc, table.long(), n)
    with pytest.raises(ValueError):
        paged_decode(q, kc, vc, table, torch.tensor([20, 1], dtype=torch.int32, device=dev))
    with pytest.raises(KDAError):
        paged_decode(q[:, :3].contiguous(), kc, vc, table, n)              # 3 query heads over 2
    with pytest.raises(KDAError):
        paged_decode(q, kc[:, :, :12].contiguous(), vc[:, :, :12].contiguous(), table, n)   # page size 12
    with pytest.raises(KDAError):
        paged_decode(q, kc, vc, table, n, workspace=torch.empty(64, dtype=torch.uint8, device=dev))
    k = torch.zeros(1, 2, 64, dtype=BF, device=dev)
    with pytest.raises(ValueError):
        paged_append(k, k, kc[:, :1].contiguous(), vc, table, n)
    with pytest.raises(KDAError):
        paged_append(k[:0].expand(0, 2, 64), k[:0], kc, vc, table, n)      # one token per sequence, none given


@pytest.mark.parametrize("d,G", [(128, 4), (64, 20)])
def test_query_rows_off_16_byte_boundaries(d, G):
    dev = need_gpu()
    lens = [300, 77]
    q, kc, vc, table = _cache(lens, 2, G, d, 16, BF, seed=15)
    wide = torch.zeros(2, 2 * G * d + 5, dtype=BF, device=dev)
    wide[:, 3:3 + 2 * G * d] = q.reshape(2, -1).to(dev)
    view = wide[:, 3:3 + 2 * G * d].unflatten(1, (2 * G, d))
    n = torch.tensor(lens, dtype=torch.int32, device=dev)
    out, lse = paged_decode(view, kc.to(dev), vc.to(dev), table.to(dev), n, return_lse=True)
    ro, rl = ref.paged(q, kc, vc, table, lens, d ** -0.5)
    ref.close("out", out, ro)
    ref.close("lse", lse, rl)


@pytest.mark.parametrize("ps", [8, 16, 64])
def test_one_bad_page_among_good_ones(ps):
    """A page outside the cache in the middle of a tile, V garbage in the slot that held its place before."""
    dev = need_gpu()
    lens = [512, 512]
    q, kc, vc, table = _cache(lens, 2, 4, 128, ps, BF, seed=16)
    vc[torch.isnan(vc)] = math.inf
    for j in (1, 128 // ps + 1, 3):
        table[0, j] = -1
    ro, rl = ref.paged(q, kc, vc, table, lens, 128 ** -0.5)
    out, lse = _decode(q, kc, vc, table, lens, dev)
    ref.close("out", out, ro)
    ref.close("lse", lse, rl)
