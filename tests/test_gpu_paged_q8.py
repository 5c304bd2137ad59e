"""The paged key-value cache in 8 bits: kda_paged_append_q8 and kda_paged_decode_q8 against float64."""
import math

import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import KDAError, check_device_status, kda, paged_append_q8, paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _table(need, P, cols, seed):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(P, generator=g).tolist()
    t = torch.full((len(need), cols), -1, dtype=torch.int32)
    for i, n in enumerate(need):
        for j in range(n):
            t[i, j] = ids.pop()
    return t


def _codes(P, H, ps, d, B, seed, scales=None):
    """Random codes, some of them small, and scales of their blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(P, H, ps, d, generator=g) * torch.exp2(torch.randint(-8, 7, (P, H, ps, 1), generator=g).float())
    s = torch.exp2(torch.randint(-6, 4, (P, H, ps // B), generator=g).float()) if scales is None else scales
    return x.to(E4M3), s


def _append(k, v, kc, vc, ks, vs, table, start, lens, dev, one=False, status=None, fused=False):
    """Runs the call and the plain form on copies of the same cache; checks every code and scale."""
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        c, s = c.double(), s.double()
        ref.append(x, c, s, table, start, lens)
        want += [c, s]
    kd, vd = layers_ref.fused_rows([k, v], dev) if fused else (k.to(dev), v.to(dev))
    got = [t.to(dev) for t in (kc, ks, vc, vs)]
    cu = None if one else _i32([0] + torch.tensor(lens).cumsum(0).tolist(), dev)
    paged_append_q8(kd, vd, got[0], got[2], got[1], got[3], table.to(dev), _i32(start, dev), cu_seqlens=cu, status=status)
    torch.cuda.synchronize()
    for name, a, b in zip(("k codes", "k scales", "v codes", "v scales"), got, want):
        ref.same(name, a, b)
    return got


def _case(dtype, H, d, ps, B, lens, start, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    need = [-(-(a + n) // ps) for a, n in zip(start, lens)]
    P = sum(need) + 2
    table = _table(need, P, max(need + [0]) + 1, seed)
    T = sum(lens)
    k, v = ((torch.randn(T, H, d, generator=g) * torch.exp(spread * torch.randn(T, H, 1, generator=g))).to(dtype) for _ in range(2))
    kc, ks = _codes(P, H, ps, d, B, seed + 1)
    vc, vs = _codes(P, H, ps, d, B, seed + 2)
    return k, v, kc, vc, ks, vs, table


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ps,B", [(16, 16), (64, 16), (32, 32), (64, 64), (128, 128), (256, 32)])
def test_append(dtype, d, ps, B):
    """Ragged prompts, some from inside a block on, one empty, one of a single token."""
    dev = need_gpu()
    lens, start = [37, 0, 1, 130, 16, 5, 70], [0, 3, 17, 9, 16, 15, 120]
    _append(*_case(dtype, 3, d, ps, B, lens, start, d + ps + B), start, lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,B", [(128, 16), (64, 64), (32, 32)])
def test_append_one_token_each(dtype, d, B):
    dev = need_gpu()
    n = 37
    start = [(7 * i) % 130 for i in range(n)]
    _append(*_case(dtype, 2, d, 64, B, [1] * n, start, d), start, [1] * n, dev, one=True)
    _append(*_case(dtype, 1, d, 64, B, [1] * n, start, d + 1), start, [1] * n, dev, one=False)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_rows_of_a_wider_product(dtype):
    dev = need_gpu()
    lens, start = [20, 33], [5, 0]
    _append(*_case(dtype, 2, 64, 32, 16, lens, start, 5), start, lens, dev, fused=True)


def test_append_rows_off_16_bytes():
    dev = need_gpu()
    lens, start, H, d = [20, 33], [5, 0], 2, 64
    for dtype in (BF, F32):
        k, v, kc, vc, ks, vs, table = _case(dtype, H, d, 32, 32, lens, start, 6)
        want = []
        for x, c, s in ((k, kc, ks), (v, vc, vs)):
            c, s = c.double(), s.double()
            ref.append(x, c, s, table, start, lens)
            want += [c, s]
        flat = torch.zeros(53, 2 * H * d + 3, dtype=dtype, device=dev)
        flat[:, 1:1 + H * d], flat[:, 2 + H * d:2 + 2 * H * d] = k.flatten(1).to(dev), v.flatten(1).to(dev)
        got = [t.to(dev) for t in (kc, ks, vc, vs)]
        paged_append_q8(flat[:, 1:1 + H * d].unflatten(1, (H, d)), flat[:, 2 + H * d:2 + 2 * H * d].unflatten(1, (H, d)), got[0],
                        got[2], got[1], got[3], table.to(dev), _i32(start, dev), cu_seqlens=_i32([0, 20, 53], dev))
        for a, b in zip(got, want):
            ref.same("rows off 16 bytes", a, b)


def test_append_special_values():
    """Zeros, subnormal and huge numbers, infinities, NaN, ties, and largest values at and next to 448 times a power of two."""
    dev = need_gpu()
    d, ps = 32, 16
    up = lambda x: float(torch.nextafter(torch.tensor(x), torch.tensor(math.inf)))  # noqa: E731
    rows = [[0.0] * d, [1e-45] * d, [2.0 ** -140, -2.0 ** -130] + [0.0] * 30, [3e38, -1.0] * 16, [448.0, 1.0] * 16,
            [up(448.0), 1.0] * 16, [448.0 * 2.0 ** 50] * d, [up(448.0 * 2.0 ** -30)] * d, [math.inf, 5.0] + [1.0] * 30,
            [-math.inf, math.nan] + [0.5] * 30, [math.nan] * d, [17.0, 19.0, 21.0, 23.0, -17.0, 448.0] + [2.0 ** -9] * 26,
            [2.0 ** -10, 2.0 ** -9 * 1.5, 2.0 ** -10 * 1.01, 256.0] + [0.0] * 28, [-0.0] * d, [1.0625, 1.1875, 447.0] + [0.1] * 29]
    k = torch.tensor(rows, dtype=F32)[:, None]
    n = len(rows)
    kc, ks = _codes(n + 1, 1, ps, d, 16, 1)
    table = torch.arange(n, dtype=torch.int32)[:, None].contiguous()
    _append(k, k.flip(0).contiguous(), kc, kc, ks, ks, table, [0] * n, [1] * n, dev, one=True)
    # the same rows in one block: what is not finite leaves its neighbours' scale alone
    kc, ks = _codes(2, 1, ps, d, 16, 2)
    _append(k, k.flip(0).contiguous(), kc, kc, ks, ks, table[1:2], [0], [n], dev)
    some = torch.cat([k[8:11], k[14:15]])
    _append(some, some, kc, kc, ks, ks, table[1:2], [0], [4], dev)


def test_append_scale_of_a_partly_filled_block():
    """Kept where it is enough, grown where not, begun afresh at the block's start; one that is no power of two is rounded
    up, and one that no call can have left is recorded and its codes stay."""
    dev = need_gpu()
    H, d, ps, B = 1, 64, 32, 16
    P = 9
    scales = torch.tensor([1.0, 2.0 ** -20, 2.0 ** 100, 0.3, 5.0, math.nan, 0.0, math.inf, -1.0])[:, None, None].expand(P, H, 2).contiguous()
    kc, ks = _codes(P, H, ps, d, B, 3, scales)
    g = torch.Generator().manual_seed(4)
    k = torch.randn(P, H, d, generator=g)
    table = torch.arange(P, dtype=torch.int32)[:, None].contiguous()
    for at in (16, 0):                                                   # begun afresh
        _append(k, 2 * k, kc, kc, ks, ks, table, [at] * P, [1] * P, dev, one=True)
    _append(k[:5], k[:5], kc, kc, ks, ks, table[:5], [21] * 5, [1] * 5, dev, one=True)
    for i in range(5, 9):
        status = torch.zeros(4, dtype=torch.int32, device=dev)
        got = [t.clone().to(dev) for t in (kc, ks)]
        paged_append_q8(k[i:i + 1].to(dev), k[i:i + 1].to(dev), got[0], got[0].clone(), got[1], got[1].clone(),
                        table[i:i + 1].to(dev), _i32([21], dev), status=status)
        assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
        s = ref.scale_for(float(k[i].abs().max()))
        assert float(got[1][i, 0, 1]) == s
        want = kc.double()
        want[i, 0, 21] = ref.round_e4m3(k[i, 0].double() / s)
        ref.same("codes", got[0], want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,B", [(128, 128), (64, 64), (32, 32), (128, 16)])
def test_append_one_token_rescales_its_block(dtype, d, B):
    """A token anywhere in a block whose scale it outgrows, and in one that it does not."""
    dev = need_gpu()
    start = [0, 1, 5, 15, 16, 17, 31, 32, 47, 63, 64, 100, 111, 112, 126, 127]
    n = len(start)
    k, v, kc, vc, ks, vs, table = _case(dtype, 2, d, 128, B, [1] * n, start, d + B)
    ks, vs = ks * 2.0 ** -6, vs * torch.exp2(torch.arange(vs.shape[0]) % 2 * 8.0 - 6)[:, None, None]
    _append(k, v, kc, vc, ks, vs, table, start, [1] * n, dev, one=True)


def test_append_bf16_that_is_not_finite():
    """Infinities and NaN in bf16 blocks of one token, of some and of all of a block's warps."""
    dev = need_gpu()
    d, ps, n = 64, 64, 64
    g = torch.Generator().manual_seed(5)
    for B in (16, 64):
        x = torch.randn(3 * n, 1, d, generator=g).to(BF)
        x[3, 0, 7], x[20, 0, 63], x[40, 0, 0], x[41] = math.inf, -math.inf, math.nan, math.nan
        x[64:128] = math.nan
        x[130, 0, 2], x[131] = 2.0 ** -133, 3e38
        kc, ks = _codes(4, 1, ps, d, B, 2)
        table = torch.arange(3, dtype=torch.int32)[None]
        _append(x, x.flip(0).contiguous(), kc, kc, ks, ks, table, [0], [3 * n], dev)
        rows = x[[0, 3, 20, 41, 130, 131]].contiguous()
        six = torch.arange(6, dtype=torch.int32)[:, None].contiguous()
        kc, ks = _codes(6, 1, ps, d, B, 3)
        _append(rows, rows, kc, kc, ks, ks, six, [0, 17, 40, 33, 63, 5], [1] * 6, dev, one=True)


def test_append_in_pieces_and_at_once():
    """The same scales; the same codes but below 2^-6 of the scale, where re-rounding may move them by one step."""
    dev = need_gpu()
    H, d, ps, B, n = 2, 64, 32, 32, 75
    k, v, kc, vc, ks, vs, table = _case(BF, H, d, ps, B, [n], [0], 8, spread=3.0)
    def cache():
        return [t.to(dev) for t in (kc, vc, ks, vs)]
    whole, pieces = cache(), cache()
    kd, vd, td = k.to(dev), v.to(dev), table.to(dev)
    paged_append_q8(kd, vd, *whole, td, _i32([0], dev), cu_seqlens=_i32([0, n], dev))
    at = 0
    for m in (1, 1, 5, 30, 1, 2, 20, 15):
        paged_append_q8(kd[at:at + m], vd[at:at + m], *pieces, td, _i32([at], dev), cu_seqlens=_i32([0, m], dev))
        at += m
    assert at == n
    for c in (0, 1):
        assert torch.equal(whole[2 + c], pieces[2 + c])
        a, b = whole[c].cpu().double(), pieces[c].cpu().double()
        assert torch.equal(a[b.abs() > 2.0 ** -6], b[b.abs() > 2.0 ** -6])
        assert float((a - b).abs().max()) <= 2.0 ** -9


def test_append_malformed():
    """Bad pages, starts and offsets are recorded and skipped; nothing else changes, and the others are written."""
    dev = need_gpu()
    H, d, ps, B = 2, 64, 16, 16
    k, v, kc, vc, ks, vs, table = _case(BF, H, d, ps, B, [20, 20, 20], [0, 5, 0], 9)
    P = kc.shape[0]

    def run(table, start, cu):
        status = torch.zeros(4, dtype=torch.int32, device=dev)
        got = [t.to(dev) for t in (kc, vc, ks, vs)]
        paged_append_q8(k.to(dev), v.to(dev), *got, table.to(dev), _i32(start, dev), cu_seqlens=_i32(cu, dev), status=status)
        return got, check_device_status(status)

    bad = table.clone()
    bad[0, 1], bad[1, 0], bad[2, 1] = P, -1, -7
    got, st = run(bad, [0, 5, 0], [0, 20, 40, 60])
    assert st == kda.KDA_ERR_INVALID_ARG
    want = [t.double() for t in (kc, vc, ks, vs)]
    for x, c, s in ((k, want[0], want[2]), (v, want[1], want[3])):
        ref.append(x[:16], c, s, table[:1], [0], [16])
        ref.append(x[31:40], c, s, table[1:2], [16], [9])
        ref.append(x[40:56], c, s, table[2:], [0], [16])
    for a, b in zip(got, want):
        ref.same("bad pages", a, b)
    cols = table.shape[1] * ps
    # (with the last offsets the second sequence has 40 tokens, and pages for 27 of them)
    for start, cu, n in (([-1, 5, 0], [0, 20, 40, 60], 20), ([cols, 5, 0], [0, 20, 40, 60], 20),
                         ([2 ** 31 - 1, 5, 0], [0, 20, 40, 60], 20), ([0, 5, 0], [20, 0, 40, 60], 27)):
        got, st = run(table, start, cu)
        assert st == kda.KDA_ERR_INVALID_ARG
        want = [t.double() for t in (kc, vc, ks, vs)]
        for x, c, s in ((k, want[0], want[2]), (v, want[1], want[3])):
            ref.append(x[cu[1]:cu[1] + n], c, s, table[1:2], [5], [n])
            ref.append(x[40:60], c, s, table[2:], [0], [20])
        for a, b in zip(got, want):
            ref.same("bad start or offsets", a, b)
    assert run(table, [0, 5, 0], [0, 20, 40, 59])[1] == kda.KDA_ERR_INVALID_ARG
    got, st = run(table, [0, 5, 0], [0, 20, 40, 61])
    assert st == kda.KDA_ERR_INVALID_ARG


# ------------------------------------------------------------------------------------------------ decode
def _cache(lens, H, G, d, ps, B, dtype, seed, scales=None, extra=1):
    """Random pages; codes that no token was written to are NaN, scales of blocks without any too."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // ps) for n in lens]
    P = sum(need) + 2
    table = _table(need, P, max(need + [0]) + extra, seed)
    kc, ks = _codes(P, H, ps, d, B, seed + 1)
    vc, vs = _codes(P, H, ps, d, B, seed + 2)
    kc, vc = ((torch.randn(P, H, ps, d, generator=g) * 100).to(E4M3) for _ in range(2))
    if scales is None:
        ks, vs = (torch.exp2(torch.randint(-8, -5, (P, H, ps // B), generator=g).float()) for _ in range(2))
    else:
        ks, vs = scales(P, H, ps // B, g)
    used = torch.zeros(P, ps, dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(need[i]):
            used[int(table[i, j]), :min(ps, n - j * ps)] = True
    for c, s in ((kc, ks), (vc, vs)):
        c.view(torch.uint8).masked_fill_(~used[:, None, :, None], 0x7F)
        s.masked_fill_(~used.unflatten(1, (-1, B)).any(-1)[:, None], math.nan)
    q = torch.randn(len(lens), H * G, d, generator=g).to(dtype)
    return q, kc, vc, ks, vs, table


def _same(a, b):
    """Bit for bit, NaN in the same places (a few of the random codes are)."""
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


def _decode(c, lens, dev, scale=None, check=True, **kw):
    q, kc, vc, ks, vs, table = c
    out, lse = paged_decode_q8(*(t.to(dev) for t in c), _i32(lens, dev), scale=scale, return_lse=True, **kw)
    if check:
        ro, rl = ref.decode(q, kc, vc, ks, vs, table, lens, q.shape[2] ** -0.5 if scale is None else scale)
        ref.close("out", out, ro)
        layers_ref.close("lse", lse, rl)
    return out, lse


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("ps,B,G", [(16, 16, 4), (64, 16, 1), (32, 32, 8), (128, 64, 3), (256, 128, 12)])
def test_decode(dtype, d, ps, B, G):
    """Lengths from none to several tiles, pages that end inside a tile and tiles inside a page."""
    dev = need_gpu()
    lens = [130, 0, 1, 15, 16, 17, 128, 257, 600, 127]
    _decode(_cache(lens, 2, G, d, ps, B, dtype, d + G), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("G", [1, 2, 5, 7, 8, 9, 16, 17, 32, 40])
def test_decode_heads(dtype, G):
    dev = need_gpu()
    lens = [200, 33, 5]
    _decode(_cache(lens, 1, G, 64, 32, 16, dtype, G), lens, dev)
    _decode(_cache(lens, 3, G, 128, 16, 16, dtype, G + 1), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_one_long_row(dtype):
    dev = need_gpu()
    lens = [20011]
    _decode(_cache(lens, 2, 4, 128, 64, 16, dtype, 1), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_many_rows(dtype):
    dev = need_gpu()
    lens = [(37 * i) % 300 for i in range(300)]
    _decode(_cache(lens, 2, 4, 64, 16, 16, dtype, 2), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_any_scales(dtype):
    """Scales that are no powers of two, negative or zero, and of very different size from block to block."""
    dev = need_gpu()
    lens = [300, 40, 129]
    def odd(P, H, n, g):
        return ((torch.rand(P, H, n, generator=g) - 0.3) / 50 for _ in range(2))
    def wide(P, H, n, g):
        return (torch.exp2(torch.randint(-20, -6, (P, H, n), generator=g).float()) * s for s in (1.0, 2.0 ** 60))
    def none(P, H, n, g):
        return torch.full((P, H, n), 0.01), torch.zeros(P, H, n)
    for scales in (odd, wide):
        _decode(_cache(lens, 2, 4, 128, 32, 16, dtype, 3, scales), lens, dev)
    out, _ = _decode(_cache(lens, 2, 4, 128, 32, 16, dtype, 3, none), lens, dev)
    assert not out.nan_to_num().any()                                    # (a code of the cache is NaN, as checked against the plain form)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_queries_of_any_size(dtype):
    """Tiny, huge and zero queries, and channels of very different size in one head."""
    dev = need_gpu()
    lens = [200, 70, 9, 30]
    c = _cache(lens, 2, 4, 64, 32, 16, dtype, 4)
    q = c[0].float()
    q[0] *= 2.0 ** -100
    q[1] *= 2.0 ** 20
    q[2] = 0
    q[3, :, ::7] *= 2.0 ** 12
    c = (q.to(dtype), *c[1:])
    _decode(c, lens, dev, scale=2.0 ** -24)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_own_and_others_values(dtype):
    """NaN in a row's own tokens gives NaN in its heads alone; a query's infinity or NaN stays in its head."""
    dev = need_gpu()
    lens = [200, 150, 90]
    c = _cache(lens, 2, 4, 64, 32, 16, dtype, 5)
    plain, _ = _decode(c, lens, dev)
    q, kc, vc, ks, vs, table = (t.clone() for t in c)
    kc.view(torch.uint8)[int(table[0, 2]), 0, 3, 5] = 0x7F
    vc.view(torch.uint8)[int(table[1, 1]), 1, 3, 7] = 0xFF
    q[2, 1, 4] = math.inf
    q[2, 6, 4] = math.nan
    out, _ = _decode((q, kc, vc, ks, vs, table), lens, dev, check=False)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, :4], bad[1, 4:, 7], bad[2, 1], bad[2, 6] = True, True, True, True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], plain[~bad])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_bad_pages_and_lengths(dtype):
    dev = need_gpu()
    lens = [200, 100, 64, 300]
    q, kc, vc, ks, vs, table = _cache(lens, 2, 2, 64, 32, 16, dtype, 6)
    table[0, 1], table[1, 0], table[2, 0], table[2, 1] = -1, kc.shape[0], -1, 1 << 30
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    out, lse = _decode((q, kc, vc, ks, vs, table), lens, dev, status=status)
    assert not out[2].any() and torch.isinf(lse[2]).all()
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    # past the table: its end; negative: none
    lens = [200, 100, 64, 300]
    c = _cache(lens, 2, 2, 64, 32, 16, dtype, 7, extra=0)
    cols = c[5].shape[1] * 32
    status.zero_()
    c[5][3] = torch.randperm(c[1].shape[0], generator=torch.Generator().manual_seed(0))[:cols // 32].to(torch.int32)
    for s in c[1:3]:
        s.view(torch.uint8).masked_fill_(torch.isnan(s.float()), 0x30)
    for s in c[3:5]:
        s.nan_to_num_(0.01)
    out, lse = paged_decode_q8(*(t.to(dev) for t in c), _i32([200, -5, 64, 1 << 30], dev), return_lse=True, status=status)
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    ro, rl = ref.decode(*c, [200, 0, 64, cols], 64 ** -0.5)
    ref.close("out", out, ro)
    layers_ref.close("lse", lse, rl)


FORMS = [(32, 3), (32, 16), (32, 20), (64, 8), (64, 11), (64, 33), (128, 8), (128, 16), (128, 24)]


@pytest.mark.parametrize("d,G", FORMS)
@pytest.mark.parametrize("ps,B", [(1024, 128), (1024, 16), (16, 16), (128, 32)])
def test_decode_lengths_of_every_form(d, G, ps, B):
    """Rows of one and two tokens, that end next to a tile's, a page's and a block's end, and a row without any."""
    dev = need_gpu()
    lens = [1, 2, 0, 15, 17, 127, 128, 129, 255, 256, 257, 511, 513, 1023, 1025, 31]
    _decode(_cache(lens, 1, G, d, ps, B, BF, d + G + ps), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,G", FORMS)
def test_decode_missing_pages_of_every_form(dtype, d, G):
    """Pages that are missing at the front, in the middle and at the end of a tile, several in a row, and all of a tile."""
    dev = need_gpu()
    lens = [700, 600, 520, 90, 530]
    q, kc, vc, ks, vs, table = _cache(lens, 2, G, d, 16, 16, dtype, d + G)
    P = kc.shape[0]
    for row, cols in enumerate(([0], [3, 4, 5, 31], range(16, 33), range(6), [1, 2, 7, 8, 15, 16, 32, 33])):
        for i in cols:
            table[row, i] = (-1, P, 1 << 30, -2 ** 31)[i % 4]
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    out, lse = _decode((q, kc, vc, ks, vs, table), lens, dev, status=status)
    assert not out[3].any() and torch.isneginf(lse[3]).all()
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,G", FORMS)
def test_decode_values_of_their_own_of_every_form(dtype, d, G):
    """NaN in a row's own tokens, next to others' in a row of the tile, stays in that row's heads and channels."""
    dev = need_gpu()
    lens = [200, 150, 90, 60]
    c = _cache(lens, 2, G, d, 32, 16, dtype, d + G + 1)
    plain, _ = _decode(c, lens, dev)
    q, kc, vc, ks, vs, table = (t.clone() for t in c)
    kc.view(torch.uint8)[int(table[0, 2]), 0, 3, 5] = 0x7F
    vc.view(torch.uint8)[int(table[1, 1]), 1, 4, 7] = 0xFF
    vc.view(torch.uint8)[int(table[3, 1]), 0, 27, d - 1] = 0x7F          # the last token
    q[2, 1, 4] = math.inf
    q[2, 2 * G - 1, d - 1] = math.nan
    out, _ = _decode((q, kc, vc, ks, vs, table), lens, dev, check=False)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[0, :G], bad[1, G:, 7], bad[2, 1], bad[2, 2 * G - 1], bad[3, :G, d - 1] = True, True, True, True, True
    bad |= torch.isnan(plain)                                            # (a few of the random codes are NaN)
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], plain[~bad])


@pytest.mark.parametrize("d,G", FORMS)
def test_decode_many_short_rows_of_every_form(d, G):
    """Items of one tile and of a few, whole and cut, more of them than CTAs."""
    dev = need_gpu()
    g = torch.Generator().manual_seed(d + G)
    lens = [int(n) for n in torch.randint(0, 700, (90,), generator=g)]
    _decode(_cache(lens, 2, G, d, 64, 32, BF, d + G + 2), lens, dev)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decode_query_rows_of_a_wider_product(dtype):
    dev = need_gpu()
    lens = [100, 33, 257]
    c = _cache(lens, 2, 4, 64, 32, 32, dtype, 8)
    plain, _ = _decode(c, lens, dev)
    flat = torch.zeros(3, 8 * 64 + 5, dtype=dtype, device=dev)
    for at in (0, 1):
        flat[:, at:at + 8 * 64] = c[0].flatten(1).to(dev)
        rest = [t.to(dev) for t in c[1:]]
        assert _same(paged_decode_q8(flat[:, at:at + 512].unflatten(1, (8, 64)), *rest, _i32(lens, dev)), plain)


def test_no_rows_no_pages():
    dev = need_gpu()
    q = torch.zeros(0, 4, 64, dtype=BF, device=dev)
    kc = torch.zeros(3, 2, 16, 64, dtype=torch.uint8, device=dev).view(E4M3)
    ks = torch.ones(3, 2, 1, device=dev)
    assert paged_decode_q8(q, kc, kc, ks, ks, _i32([], dev).reshape(0, 2), _i32([], dev)).shape == (0, 4, 64)
    q = torch.ones(2, 4, 64, dtype=BF, device=dev)
    none = kc[:0]
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    out, lse = paged_decode_q8(q, none, none, ks[:0], ks[:0], _i32([[0], [0]], dev), _i32([0, 3], dev), return_lse=True, status=status)
    assert not out.any() and torch.isinf(lse).all()
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG


def test_results_do_not_depend_on_the_run():
    dev = need_gpu()
    lens = [5000, 1, 300, 2222]
    c = [t.to(dev) for t in _cache(lens, 2, 4, 128, 64, 16, BF, 9)]
    first = paged_decode_q8(*c, _i32(lens, dev), return_lse=True)
    for _ in range(5):
        again = paged_decode_q8(*c, _i32(lens, dev), return_lse=True)
        assert all(_same(a, b) for a, b in zip(first, again))


def test_refusals():
    dev = need_gpu()
    lens = [20]
    q, kc, vc, ks, vs, table = (t.to(dev) for t in _cache(lens, 2, 2, 64, 32, 16, BF, 10))
    n = _i32(lens, dev)
    with pytest.raises(TypeError):
        paged_decode_q8(q, kc.view(torch.uint8), vc, ks, vs, table, n)
    with pytest.raises(TypeError):
        paged_decode_q8(q.half(), kc, vc, ks, vs, table, n)
    with pytest.raises(ValueError):
        paged_decode_q8(q, kc, vc, ks[:, :, :1], vs, table, n)
    with pytest.raises(ValueError):
        paged_decode_q8(q, kc, vc, ks.repeat(1, 1, 2)[:, :, :3].contiguous(), vs, table, n)
    with pytest.raises(KDAError):                                        # blocks of 8 tokens
        paged_decode_q8(q, kc, vc, ks.repeat(1, 1, 2), vs.repeat(1, 1, 2), table, n)
    with pytest.raises(ValueError):
        paged_decode_q8(q, kc.cpu(), vc, ks, vs, table, n)
    k = torch.zeros(1, 2, 64, dtype=BF, device=dev)
    with pytest.raises(TypeError):
        paged_append_q8(k, k.float(), kc, vc, ks, vs, table, n)
    with pytest.raises(ValueError):
        paged_append_q8(k, k, kc, vc, ks, vs, table, n[:0])
    with pytest.raises(TypeError):
        paged_append_q8(k, k, kc, vc, ks.double(), vs, table, n)
