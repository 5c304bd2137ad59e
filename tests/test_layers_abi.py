"""Host-side checks of include/kda_layers.h and of its binding, without a GPU."""
import ctypes

import pytest
import torch

from gated_delta_rule_46_gb300 import kda, layers

BF, F32 = kda.KDA_BF16, kda.KDA_F32
INV, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
A = 4096            # an address that no check dereferences


def _linear(**kw):
    a = dict(x=A, ldx=64, w=A, bias=A, residual=A, out=A, M=4, N=8, K=64, act=0, dt=BF, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_linear")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(M=-1), INV), (dict(K=0), INV), (dict(ldx=63), INV), (dict(act=5), UNS),
                                     (dict(act=-1), UNS), (dict(dt=3), UNS), (dict(x=None), INV), (dict(out=A + 1), INV),
                                     (dict(residual=A + 1), INV), (dict(bias=A + 2), INV), (dict(M=0, x=None), OK),
                                     (dict(N=0), OK), (dict(N=1 << 31), UNS)])
def test_linear(kw, want):
    assert _linear(**kw) == want


def _prefill(**kw):
    a = dict(q=A, ldq=256, k=A, ldk=256, v=A, ldv=256, ld=A, cu=A, n=1, T=8, H=2, dk=128, dv=128, dt=BF, scale=1.0, s0=None,
             s1=None, out=A, ws=None, wsb=0, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_decay_prefill")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(n=-1), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(dk=96), UNS),
                                     (dict(dt=9), UNS), (dict(ldq=255), INV), (dict(ldv=255), INV), (dict(n=0, q=None), OK),
                                     (dict(cu=None), INV), (dict(ld=None), INV), (dict(v=None), INV), (dict(s0=A + 4), INV),
                                     (dict(ws=A + 8), INV), (dict(q=A + 1), INV), (dict(T=1 << 31), UNS)])
def test_decay_prefill(kw, want):
    assert _prefill(**kw) == want


def _decode(**kw):
    a = dict(q=A, ldq=256, k=A, ldk=256, v=A, ldv=256, ld=A, pool=A, P=4, slots=A, out=A, N=3, H=2, dk=128, dv=128, dt=BF,
             scale=1.0, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_decay_decode")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(N=-1), INV), (dict(P=-1), INV), (dict(slots=None, P=2), INV), (dict(dv=48), UNS),
                                     (dict(pool=A + 4), INV), (dict(pool=None), INV), (dict(ldk=255), INV), (dict(N=0), OK)])
def test_decay_decode(kw, want):
    assert _decode(**kw) == want


def _append(**kw):
    a = dict(k=A, ldk=256, v=A, ldv=256, kc=A, vc=A, P=9, ps=16, table=A, cols=4, start=A, cu=A, n=3, T=7, H=2, d=128, dt=BF,
             status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_paged_append")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(ps=0), UNS), (dict(ps=12), UNS), (dict(ps=2048), UNS), (dict(d=80), UNS),
                                     (dict(cu=None), INV), (dict(ldk=10), INV), (dict(kc=A + 2), INV), (dict(table=None), INV),
                                     (dict(T=0), OK), (dict(n=0), OK), (dict(cols=-1), INV), (dict(H=0), INV)])
def test_paged_append(kw, want):
    assert _append(**kw) == want


def _attend(**kw):
    a = dict(q=A, ldq=1024, kc=A, vc=A, P=9, ps=16, table=A, cols=4, lens=A, n=3, Hq=8, Hkv=2, d=128, dt=BF, scale=1.0, out=A,
             lse=None, ws=A, wsb=1 << 30, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_paged_decode")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(Hq=7), INV), (dict(Hkv=0), INV), (dict(ps=24), UNS), (dict(d=16), UNS),
                                     (dict(ws=None), INV), (dict(wsb=16), INV), (dict(lens=None), INV), (dict(ldq=1023), INV),
                                     (dict(n=0), OK), (dict(table=None), INV), (dict(vc=A + 8), INV), (dict(dt=2), UNS),
                                     (dict(cols=1 << 28, ps=16), UNS)])
def test_paged_decode(kw, want):
    assert _attend(**kw) == want


def test_workspace_sizes():
    ws = layers.paged_decode_workspace_size
    assert ws(4, 1000, 8, 2, 128) > 0 and ws(4, 1000, 8, 2, 128) % 256 == 0
    assert ws(4, 1000, 8, 3, 128) == 0 and ws(0, 1000, 8, 2, 128) == 0
    assert ws(1, 64, 2, 2, 64) < ws(4, 1 << 20, 8, 2, 128) == ws(4, 1 << 24, 8, 2, 128)
    assert layers.decay_prefill_workspace_size(64, 1, 2, 32, 32, torch.float32) % 16 == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        layers.linear(x, x)
    with pytest.raises(ValueError):
        layers.decay_prefill(q, q, q, torch.zeros(2), i)
    with pytest.raises(ValueError):
        layers.decay_decode(q, q, q, torch.zeros(2), torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError):
        layers.paged_append(q, q, c, c, i[:, None], i)
    with pytest.raises(ValueError):
        layers.paged_decode(q, c, c, i[:, None], i)


def test_row_strides():
    """The binding's row-stride rule: dense rows pass with their stride, others are refused."""
    t = torch.zeros(5, 40)
    rows = lambda x: layers._rows(x, "t", tuple(x.shape), x.shape[1:].numel(), torch.float32, x.device)  # noqa: E731
    assert rows(t) == 40 and rows(t[:, 8:24]) == 40 and rows(t[:, 8:24].unflatten(1, (2, 8))) == 40
    assert rows(t[:0]) == 40 and rows(t[::2]) == 80 and rows(t[:1, :8]) >= 8
    for bad in (t.t(), t[:, ::2], t[:, None, :8].expand(5, 3, 8), t[:1].expand(5, 40)):
        with pytest.raises(ValueError):
            rows(bad)


def test_addresses_are_not_truncated():
    """Every pointer argument is declared as a pointer, every size as 64 bits."""
    for name, (_, args) in layers._SIGNATURES.items():
        assert all(a in (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t) for a in args), name
