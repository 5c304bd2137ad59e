"""Softmax weights of kda_paged_decode_q8 where scores are peaked and blocks of V of very different size.

A token's weight here is w = e^{s - max s} |v_scale|.  For bf16 queries it is rounded to two e4m3 parts: off by at most
2^-8 of itself, or 2^-21 of the largest of its tile (128 or 256 tokens from the row's start on: the largest of a window of
256 is no smaller).  Each token's value lies in one channel, so that a channel sums a token or a few, and the bound holds for
every output by itself:
    |out - ref| <= sum (2^-8 w + 2^-21 max w) |code| / l + 2^-8 |out|.
Scores of up to 24 (35 in base 2) are off by 2^-19 in float32, and sums and exponentials by less than that a step: 2^-15 of a
weight covers them, and the rounding to float16 before the parts are split is 2^-11 of it.  Queries are powers of two and
their products with the codes exact.  For float32 queries 2^-15 is all there is.
"""
import math

import pytest
import torch

import cache8_ref as ref
import layers_ref
from gated_delta_rule_46_gb300 import paged_decode_q8
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3
FORMS = [(32, 3), (32, 16), (32, 20), (64, 8), (64, 11), (64, 33), (128, 8), (128, 16), (128, 24)]
LENS = [100, 256, 700, 1, 37]
PS, B, H = 32, 16, 2
KINDS = ["equal", "sink", "first small", "first large", "wide", "wider", "any", "zero blocks", "tiny", "missing pages"]


def _case(kind, dtype, d, G, seed):
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // PS) for n in LENS]
    P, cols = sum(need) + 1, max(need)
    ids = torch.randperm(P, generator=g).to(torch.int32).tolist()
    table = torch.full((len(LENS), cols), -1, dtype=torch.int32)
    k, v = torch.zeros(P, H, PS, d), torch.zeros(P, H, PS, d)
    ks, vs = torch.ones(P, H, PS // B), torch.full((P, H, PS // B), 2.0 ** -5)
    for i, n in enumerate(LENS):
        for j in range(need[i]):
            table[i, j] = ids.pop()
        for h in range(H):
            gap = torch.linspace(0, 16, n)[torch.randperm(n, generator=g)]               # nats below the largest score
            chan = torch.randperm(n, generator=g) % d
            if kind == "sink":                           # the first token takes nearly all of the weight, and its value is 0
                gap, gap[0] = 8 + gap / 2, 0.0
            if kind.startswith("first"):
                gap, gap[0] = 10 + gap / 4, 0.0
            for t in range(n):
                p, o = int(table[i, t // PS]), t % PS
                big = float(ref.round_e4m3(gap[t].double()))
                k[p, h, o, 0], k[p, h, o, 1] = -big, big - float(gap[t])
                v[p, h, o, chan[t]] = float(torch.randint(8, 16, (), generator=g)) * (0.0 if kind == "sink" and t == 0 else 1.0)
    shape = vs.shape
    if kind in ("wide", "missing pages"):
        vs = torch.exp2(torch.randint(-18, 1, shape, generator=g).float())
    elif kind == "wider":
        vs = torch.exp2(torch.randint(-60, 60, shape, generator=g).float())
    elif kind == "any":
        vs = (torch.rand(shape, generator=g) - 0.5) * torch.exp2(torch.randint(-9, 1, shape, generator=g).float())
    elif kind == "zero blocks":
        vs = vs * (torch.rand(shape, generator=g) < 0.5)
    elif kind == "tiny":                                 # the scales of values next to the smallest normal number
        vs = torch.exp2(torch.randint(-126, -118, shape, generator=g).float())
    elif kind in ("first small", "first large"):
        vs = vs * torch.exp2(torch.randint(-1, 1, shape, generator=g).float())
        for i in range(len(LENS)):
            vs[int(table[i, 0]), :, 0] = 2.0 ** (-17 if kind == "first small" else 3)
    if kind == "missing pages":
        for i, j in ((0, 1), (1, 0), (2, 5), (2, 6), (2, 20)):
            table[i, j] = -1
    # every head another steepness; powers of two
    f = torch.exp2(-(torch.arange(G * H) % 4).float())
    q = torch.zeros(len(LENS), G * H, d)
    q[:, :, 0] = q[:, :, 1] = f
    return q.to(dtype), k.to(E4M3), v.to(E4M3), ks, vs, table


def _bound(case, dtype):
    """Outputs, and how far each may be off, in float64."""
    q, kc, vc, ks, vs, table = case
    N, Hq, d = q.shape
    G, V = Hq // H, vc.double()
    w_scale = vs.double().repeat_interleave(B, 2)
    K = ref.values(kc, ks)
    out, most = torch.zeros(N, Hq, d, dtype=torch.float64), torch.zeros(N, Hq, d, dtype=torch.float64)
    for i, n in enumerate(LENS):
        pos = torch.tensor([t for t in range(n) if table[i, t // PS] >= 0], dtype=torch.long)
        if not len(pos):
            continue
        p, o = table[i].long()[pos // PS], pos % PS
        for hq in range(Hq):
            h = hq // G
            s = K[p, h, o] @ q[i, hq].double()
            e = torch.exp(s - s.max())
            u = w_scale[p, h, o]
            w, codes = e * u, V[p, h, o]
            top = torch.zeros(n // 256 + 1, dtype=torch.float64).scatter_reduce(0, pos // 256, w.abs(), "amax")[pos // 256]
            off = w.abs() * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -15) + 2.0 ** -21 * top if dtype is BF else w.abs() * 2.0 ** -15
            out[i, hq] = w @ codes / e.sum()
            most[i, hq] = off @ codes.abs() / e.sum()
    most += (2.0 ** -8 if dtype is BF else 2.0 ** -23) * (out.abs() + most)
    return out, most


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,G", FORMS)
def test_weights(d, G, kind, dtype):
    dev = need_gpu()
    case = _case(kind, dtype, d, G, 1000 * KINDS.index(kind) + d + G)
    want, most = _bound(case, dtype)
    got, lse = paged_decode_q8(*(t.to(dev) for t in case), torch.tensor(LENS, dtype=torch.int32, device=dev), scale=1.0,
                               return_lse=True)
    off = (got.cpu().double() - want).abs()
    if kind == "tiny":
        # products next to the smallest normal number: float32 keeps multiples of 2^-149, of each of a sum's terms; and below
        # 2^-126 a bf16 output is a multiple of 2^-133, its seven bits of fraction below that power: off by 2^-134
        most += 2.0 ** -149 * 700 * 16 + (2.0 ** -134 if dtype is BF else 0.0)
    bad = ~(off <= most)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outputs, up to {float((off / most.clamp(min=1e-300))[bad].max()):.1f} times the bound"
    q, kc, vc, ks, vs, table = case
    layers_ref.close("lse", lse, ref.decode(*case, LENS, 1.0)[1])
    assert math.isfinite(float(want.abs().max()))
