"""Linear attention with one decay per head (kda_decay_prefill, kda_decay_decode)
against the recurrence in float64."""
import math

import pytest
import torch

import layers_ref as ref
from gated_delta_rule_46_gb300 import (KDAError, check_device_status, decay_decode, decay_prefill, kda,
                                       state_slots_copy)
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _inputs(lens, H, dk, dv, dtype, seed, init=True):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lens), len(lens)
    unit = lambda x: (x / x.norm(dim=-1, keepdim=True)).to(dtype)  # noqa: E731
    return dict(q=unit(torch.randn(T, H, dk, generator=g)), k=unit(torch.randn(T, H, dk, generator=g)),
                v=torch.randn(T, H, dv, generator=g).to(dtype), ld=-torch.exp2(-8 * torch.rand(H, generator=g)),
                lens=lens, cu=torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32),
                init=0.1 * torch.randn(N, H, dk, dv, generator=g) if init else None)


def _prefill(d, dev, fused=False, **kw):
    q, k, v = (ref.fused_rows([d["q"], d["k"], d["v"]], dev) if fused else (d[n].to(dev) for n in "qkv"))
    init = None if d["init"] is None else d["init"].to(dev)
    return decay_prefill(q, k, v, d["ld"].to(dev), d["cu"].to(dev), initial_state=init, **kw)


def _check(d, out, fin, scale=1.0):
    ro, rf = ref.decay(d["q"], d["k"], d["v"], d["ld"], d["lens"], d["init"], scale)
    ref.close("out", out, ro)
    ref.close("state", fin, rf)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 64), (128, 128), (32, 128), (128, 64), (64, 32)])
@pytest.mark.parametrize("fused", [False, True])
def test_head_sizes(dtype, dk, dv, fused):
    dev = need_gpu()
    d = _inputs([70, 1, 0, 129, 31], 3, dk, dv, dtype, seed=dk + dv)
    out, fin = _prefill(d, dev, fused, scale=0.7)
    _check(d, out, fin, 0.7)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (BF, 64), (F32, 64)])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500])
def test_lengths(dtype, d_, n):
    dev = need_gpu()
    d = _inputs([n, 3, n], 2, d_, d_, dtype, seed=n, init=n % 2 == 0)
    out, fin = _prefill(d, dev)
    _check(d, out, fin)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,H", [([2500], 2), ([1024, 1900], 1), ([0, 3000, 5], 2)])
def test_few_long_chains(dtype, lens, H):
    """Chains that the call may cut into segments; slow decays, so that the start reaches the end."""
    dev = need_gpu()
    d = _inputs(lens, H, 128, 128, dtype, seed=11)
    d["ld"] = -torch.exp2(-8 - 4 * torch.rand(H, generator=torch.Generator().manual_seed(1)))
    out, fin = _prefill(d, dev)
    _check(d, out, fin)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_chains(dtype):
    dev = need_gpu()
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in torch.randint(0, 60, (90,), generator=g)]
    d = _inputs(lens, 4, 128, 128, dtype, seed=12)
    out, fin = _prefill(d, dev, fused=True)
    _check(d, out, fin)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (F32, 64)])
def test_extreme_decays(dtype, d_):
    """No decay (log 0), hardly any, total loss within a token, and none of the past at all (log -inf)."""
    dev = need_gpu()
    d = _inputs([300, 40], 5, d_, d_, dtype, seed=13)
    d["ld"] = torch.tensor([0.0, -1e-6, -3.0, -200.0, -math.inf])
    out, fin = _prefill(d, dev)
    _check(d, out, fin)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (BF, 64), (F32, 64), (F32, 128)])
def test_non_finite_inputs_stay_where_they_belong(dtype, d_):
    """A token's infinity or NaN reaches its own and later outputs of its head and sequence, nothing else:
    not earlier tokens of the same chunk, not the neighbouring sequence in the packed rows."""
    dev = need_gpu()
    lens = [90, 150, 40]
    d = _inputs(lens, 2, d_, d_, dtype, seed=14)
    clean, cfin = _prefill(d, dev)
    at = 90 + 57                                                  # token 57 of sequence 1, head 1
    for name, val in (("v", math.inf), ("v", math.nan), ("k", math.nan), ("k", -math.inf), ("q", math.nan)):
        bad = dict(d, **{name: d[name].clone()})
        bad[name][at, 1, 3] = val
        out, fin = _prefill(bad, dev)
        ok = torch.ones(out.shape[:2], dtype=torch.bool)
        ok[at:90 + 150, 1] = False
        assert torch.isfinite(out[ok.to(dev)]).all(), (name, val)
        ref.close(f"{name} {val}", out[ok.to(dev)], clean[ok.to(dev)].double(), dtype)
        assert not torch.isfinite(out[at, 1]).all(), (name, val)
        keep = torch.ones(fin.shape[:2], dtype=torch.bool)
        if name != "q":
            keep[1, 1] = False
            assert not torch.isfinite(fin[1, 1]).all()
        assert torch.equal(fin[keep.to(dev)], cfin[keep.to(dev)]), (name, val)


def test_split_and_resume_and_in_place_state():
    dev = need_gpu()
    d = _inputs([200], 3, 128, 128, BF, seed=15)
    whole, fin = _prefill(d, dev)
    state = d["init"].to(dev)
    got = []
    for a, b in ((0, 77), (77, 77), (77, 200)):
        part = {n: d[n][a:b].to(dev) for n in "qkv"}
        cu = torch.tensor([0, b - a], dtype=torch.int32, device=dev)
        o, s = decay_prefill(part["q"], part["k"], part["v"], d["ld"].to(dev), cu, initial_state=state, final_state=state)
        assert s is state
        got.append(o)
    ref.close("resumed", torch.cat(got), whole.double())
    ref.close("state", state, fin.double())


def test_without_final_state_other_stream_and_repeats():
    dev = need_gpu()
    d = _inputs([1500, 20], 2, 128, 128, BF, seed=16)
    out, fin = _prefill(d, dev)
    torch.cuda.synchronize()
    only, none = _prefill(d, dev, want_final_state=False)
    assert none is None and torch.equal(only, out)
    dv = {n: d[n].to(dev) for n in ("q", "k", "v", "ld", "cu", "init")}
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, f2 = decay_prefill(dv["q"], dv["k"], dv["v"], dv["ld"], dv["cu"], dv["init"], stream=s)
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(f2, fin)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (F32, 32)])
def test_malformed_offsets_are_reported(dtype, d_):
    dev = need_gpu()
    d = _inputs([40, 30, 20], 2, d_, d_, dtype, seed=17)
    d["cu"] = torch.tensor([0, 40, 30, 95], dtype=torch.int32)       # sequence 1 backwards, 2 past the end
    status = torch.zeros(4, dtype=torch.int32, device=dev)
    out, fin = _prefill(d, dev, status=status, out=torch.zeros(90, 2, d_, dtype=dtype, device=dev))
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    ro, rf = ref.decay(d["q"][:40], d["k"][:40], d["v"][:40], d["ld"], [40, 0, 0], d["init"])
    ref.close("out", out[:40], ro)
    ref.close("state", fin, rf)
    assert torch.count_nonzero(out[40:]) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(32, 32), (64, 128), (128, 128), (128, 32)])
@pytest.mark.parametrize("fused", [False, True])
def test_decode_steps(dtype, dk, dv, fused):
    """Four steps over pool slots with a padding row; slots not named stay as they are."""
    dev = need_gpu()
    N, H, P = 7, 3, 11
    slots = [3, 9, -1, 0, 10, 5, 6]
    g = torch.Generator().manual_seed(dk)
    pool0 = 0.1 * torch.randn(P, H, dk, dv, generator=g)
    pool = pool0.to(dev)
    want = pool0.double()
    for step in range(4):
        d = _inputs([1] * N, H, dk, dv, dtype, seed=100 + step)
        d["ld"] = -torch.exp2(-8 * torch.rand(H, generator=torch.Generator().manual_seed(3)))
        q, k, v = (ref.fused_rows([d["q"], d["k"], d["v"]], dev) if fused else (d[n].to(dev) for n in "qkv"))
        out = decay_decode(q, k, v, d["ld"].to(dev), pool, torch.tensor(slots, dtype=torch.int32, device=dev), scale=0.5)
        ro = torch.zeros(N, H, dv, dtype=torch.float64)
        for i, s in enumerate(slots):
            if s >= 0:
                o, f = ref.decay(d["q"][i:i + 1], d["k"][i:i + 1], d["v"][i:i + 1], d["ld"], [1], want[s:s + 1], 0.5)
                ro[i], want[s] = o[0], f[0]
        ref.close("out", out, ro)
    ref.close("pool", pool, want)
    for s in (1, 2, 4, 7, 8):
        assert torch.equal(pool[s].cpu(), pool0[s])


def test_prefill_then_decode_through_the_pool():
    """Prompts through the chunked form, their states into pool slots, then token by token: the
    recurrence over the whole sequences."""
    dev = need_gpu()
    lens, more, H, D = [37, 150, 1], 3, 2, 128
    d = _inputs([n + more for n in lens], H, D, D, BF, seed=18)
    first = d["cu"].tolist()
    pick = torch.cat([torch.arange(a, a + n) for a, n in zip(first, lens)])
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    ld = d["ld"].to(dev)
    out, fin = decay_prefill(*(d[n][pick].to(dev) for n in "qkv"), ld, cu, initial_state=d["init"].to(dev))
    pool = torch.zeros(5, H, D, D, device=dev)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device=dev)
    state_slots_copy(pool, slots, fin, to_pool=True)
    ro, rf = ref.decay(d["q"], d["k"], d["v"], d["ld"], d["lens"], d["init"])
    ref.close("prompts", out, ro[pick])
    for s in range(more):
        at = torch.tensor([a + n + s for a, n in zip(first, lens)])
        o = decay_decode(*(d[n][at].to(dev) for n in "qkv"), ld, pool, slots)
        ref.close(f"step {s}", o, ro[at])
    ref.close("states", pool[slots.long()], rf)


def test_decode_bad_slot_and_non_finite():
    dev = need_gpu()
    d = _inputs([1] * 3, 2, 64, 64, F32, seed=19)
    pool0 = torch.randn(3, 2, 64, 64, generator=torch.Generator().manual_seed(2))
    pool = pool0.to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    d["v"][1, 0, 5] = math.nan
    out = decay_decode(d["q"].to(dev), d["k"].to(dev), d["v"].to(dev), d["ld"].to(dev), pool,
                       torch.tensor([3, 2, 0], dtype=torch.int32, device=dev), status=status)
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
    assert torch.count_nonzero(out[0]) == 0
    assert torch.isnan(out[1, 0, 5]) and torch.isfinite(out[2]).all() and torch.isfinite(out[1, 1]).all()
    assert int(torch.isnan(out).sum()) == 1
    assert torch.equal(pool[1].cpu(), pool0[1])


def test_refusals():
    dev = need_gpu()
    d = {n: t.to(dev) for n, t in _inputs([8], 2, 64, 64, BF, seed=20).items() if isinstance(t, torch.Tensor)}
    args = lambda **kw: [({**d, **kw})[n] for n in ("q", "k", "v", "ld", "cu")]  # noqa: E731
    with pytest.raises(TypeError):
        decay_prefill(*args(q=d["q"].half()))
    with pytest.raises(TypeError):
        decay_prefill(*args(k=d["k"].float()))
    with pytest.raises(ValueError):
        decay_prefill(*args(v=d["v"][:4]))
    with pytest.raises(ValueError):
        decay_prefill(*args(q=d["q"].transpose(0, 1).contiguous().transpose(0, 1)))
    with pytest.raises(ValueError):
        decay_prefill(*args(ld=d["ld"][:1]))
    with pytest.raises(TypeError):
        decay_prefill(*args(cu=d["cu"].long()))
    with pytest.raises(ValueError):
        decay_prefill(*args(), initial_state=d["init"].cpu())
    with pytest.raises(KDAError):
        decay_prefill(*args(q=d["q"][..., :48].contiguous(), k=d["k"][..., :48].contiguous()))
    pool = torch.zeros(4, 2, 64, 64, device=dev)
    with pytest.raises(ValueError):
        decay_decode(d["q"], d["k"], d["v"], d["ld"], pool[:, :, :, :32])
    with pytest.raises(KDAError):
        decay_decode(d["q"], d["k"], d["v"], d["ld"], pool)             # 8 rows, 4 slots, no ids


@pytest.mark.parametrize("d_", [64, 128])
@pytest.mark.parametrize("lens,H", [([3000], 3), ([700, 0, 1800], 2), ([64 * 30 + 1], 1)])
def test_segments_of_few_chains(d_, lens, H):
    """bf16 chains cut into segments, with and without the workspace that this takes; slow decays."""
    dev = need_gpu()
    d = _inputs(lens, H, d_, d_, BF, seed=21)
    d["ld"] = -torch.exp2(-9 - 3 * torch.rand(H, generator=torch.Generator().manual_seed(4)))
    out, fin = _prefill(d, dev)
    _check(d, out, fin)
    one, last = _prefill(d, dev, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    _check(d, one, last)
    state = d["init"].to(dev)                                     # the start state's buffer takes the end state
    d["init"] = state
    again, same = _prefill(d, dev, final_state=state)
    assert same is state and torch.equal(again, out) and torch.equal(state, fin)


@pytest.mark.parametrize("dtype,dk,dv", [(F32, 128, 128), (F32, 64, 32), (BF, 32, 64), (F32, 32, 128)])
@pytest.mark.parametrize("lens,H", [([2500], 3), ([600, 0, 1500], 2), ([32 * 40 + 5], 1)])
def test_segments_on_the_cuda_cores(dtype, dk, dv, lens, H):
    dev = need_gpu()
    d = _inputs(lens, H, dk, dv, dtype, seed=22)
    d["ld"] = -torch.exp2(-9 - 3 * torch.rand(H, generator=torch.Generator().manual_seed(5)))
    out, fin = _prefill(d, dev, fused=True)
    _check(d, out, fin)
    one, last = _prefill(d, dev, workspace=torch.zeros(16, dtype=torch.uint8, device=dev))
    _check(d, one, last)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (BF, 64), (F32, 64)])
def test_unaligned_rows(dtype, d_):
    """q, k, v that start on odd elements of wider rows: no 16-byte copies possible."""
    dev = need_gpu()
    d = _inputs([100, 33], 2, d_, d_, dtype, seed=23)
    wide = {n: torch.zeros(133, 2 * d_ + 7, dtype=dtype, device=dev) for n in "qkv"}
    views = {}
    for i, n in enumerate("qkv"):
        wide[n][:, i + 1:i + 1 + 2 * d_] = d[n].reshape(133, -1).to(dev)
        views[n] = wide[n][:, i + 1:i + 1 + 2 * d_].unflatten(1, (2, d_))
    out, fin = decay_prefill(views["q"], views["k"], views["v"], d["ld"].to(dev), d["cu"].to(dev), d["init"].to(dev))
    _check(d, out, fin)


@pytest.mark.parametrize("dtype,d_", [(BF, 128), (F32, 64)])
def test_overlapping_offsets_stay_inside_the_workspace(dtype, d_):
    """Offsets that go back and forth name more tokens than there are: reported, nothing out of range."""
    dev = need_gpu()
    d = _inputs([3000], 1, d_, d_, dtype, seed=24, init=False)
    cu = [0, 3000, 0, 3000, 0, 3000, 0, 3000]
    d["cu"] = torch.tensor(cu, dtype=torch.int32)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, fin = _prefill(d, dev, status=status)
    assert check_device_status(status) == kda.KDA_ERR_INVALID_ARG
