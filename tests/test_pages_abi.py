"""Host-side checks of the cache in 8 bits and of its pages, without a GPU."""
import ctypes

import pytest
import torch

import cache8_ref as ref
from gated_delta_rule_46_gb300 import kda, layers, pages

BF = kda.KDA_BF16
INV, UNS, OK = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_OK
A = 4096            # an address that no check dereferences


def _append(**kw):
    a = dict(k=A, ldk=256, v=A, ldv=256, kc=A, vc=A, ks=A, vs=A, P=9, ps=64, B=16, table=A, cols=4, start=A, cu=A, n=3, T=7, H=2,
             d=128, dt=BF, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_paged_append_q8")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(ps=0), UNS), (dict(ps=48), UNS), (dict(ps=8), UNS), (dict(B=8), UNS), (dict(B=128), UNS),
                                     (dict(B=256, ps=256), UNS), (dict(B=24), UNS), (dict(B=0), UNS), (dict(d=80), UNS),
                                     (dict(dt=2), UNS), (dict(cu=None), INV), (dict(ldk=255), INV), (dict(kc=A + 8), INV),
                                     (dict(ks=None), INV), (dict(vs=A + 2), INV), (dict(k=A + 1), INV), (dict(table=None), INV),
                                     (dict(start=A + 1), INV), (dict(T=0), OK), (dict(n=0), OK), (dict(cols=-1), INV),
                                     (dict(H=0), INV), (dict(T=1 << 31), UNS)])
def test_paged_append_q8(kw, want):
    assert _append(**kw) == want


def _attend(**kw):
    a = dict(q=A, ldq=1024, kc=A, vc=A, ks=A, vs=A, P=9, ps=64, B=32, table=A, cols=4, lens=A, n=3, Hq=8, Hkv=2, d=128, dt=BF,
             scale=1.0, out=A, lse=None, ws=A, wsb=1 << 30, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_paged_decode_q8")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(Hq=7), INV), (dict(Hkv=0), INV), (dict(ps=24), UNS), (dict(B=64, ps=32), UNS),
                                     (dict(d=16), UNS), (dict(ws=None), INV), (dict(wsb=16), INV), (dict(lens=None), INV),
                                     (dict(ldq=1023), INV), (dict(n=0), OK), (dict(table=None), INV), (dict(ks=None), INV),
                                     (dict(vs=A + 1), INV), (dict(vc=A + 8), INV), (dict(dt=2), UNS), (dict(lse=A + 2), INV),
                                     (dict(cols=1 << 28, ps=16, B=16), UNS)])
def test_paged_decode_q8(kw, want):
    assert _attend(**kw) == want


def _resize(**kw):
    a = dict(table=A, n=4, cols=5, held=A, refs=A, P=9, tokens=A, ps=16, ws=A, wsb=1 << 20, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_pages_resize")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(n=-1), INV), (dict(P=-1), INV), (dict(ps=3), UNS), (dict(ps=2048), UNS), (dict(n=0), OK),
                                     (dict(held=None), INV), (dict(refs=None), INV), (dict(tokens=A + 2), INV),
                                     (dict(ws=A + 8), INV), (dict(wsb=4 * 70000 - 1, P=70000), INV), (dict(ws=None, P=70000), INV), (dict(table=None), INV),
                                     (dict(n=1 << 16, cols=1 << 15), UNS)])
def test_resize(kw, want):
    assert _resize(**kw) == want


def _arrays(ptrs, sizes):
    return (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(sizes))(*sizes)


def _fork(ptrs=(A, A), sizes=(64, 3), **kw):
    p, s = _arrays(ptrs, sizes)
    a = dict(pools=p, sizes=s, np=len(ptrs), table=A, n=4, cols=5, held=A, refs=A, P=9, lens=A, src=A, dst=A, f=2, ps=16, ws=A,
             wsb=1 << 20, status=None, stream=None)
    a.update(kw)
    return layers._fn("kda_pages_fork")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(f=0), OK), (dict(f=-1), INV), (dict(np=-1), INV), (dict(pools=None), INV),
                                     (dict(sizes=(64, -1)), INV), (dict(ptrs=(A, None)), INV), (dict(src=None), INV),
                                     (dict(lens=None), INV), (dict(dst=A + 1), INV), (dict(ps=17), UNS), (dict(ws=None), INV),
                                     (dict(wsb=100), INV), (dict(table=None), INV), (dict(n=1 << 16, cols=1 << 15), UNS)])
def test_fork(kw, want):
    assert _fork(**kw) == want


def _compact(ptrs=(A,), sizes=(64,), **kw):
    p, s = _arrays(ptrs, sizes)
    a = dict(pools=p, sizes=s, np=len(ptrs), table=A, n=4, cols=5, refs=A, P=9, map=A, live=A, ws=A, wsb=1 << 20, status=None,
             stream=None)
    a.update(kw)
    return layers._fn("kda_pages_compact")(*a.values())


@pytest.mark.parametrize("kw,want", [(dict(P=-1), INV), (dict(map=None), INV), (dict(live=None), INV), (dict(live=A + 1), INV),
                                     (dict(refs=None), INV), (dict(table=None), INV), (dict(ws=None), INV), (dict(wsb=16), INV),
                                     (dict(sizes=(-4,)), INV)])
def test_compact(kw, want):
    assert _compact(**kw) == want


def test_workspace_sizes():
    size = lambda name, *a: layers._fn(name)(*a)  # noqa: E731
    assert size("kda_pages_resize_workspace_size", 4, 5, 65537) >= 4 * 65537
    assert size("kda_pages_resize_workspace_size", 4, 5, 65536) == 0
    assert size("kda_pages_resize_workspace_size", 1 << 16, 1 << 15, 9) == 0
    assert size("kda_pages_fork_workspace_size", 10, 5, 7) > 0 and size("kda_pages_fork_workspace_size", 10, 5, -1) == 0
    assert size("kda_pages_compact_workspace_size", 1000) >= 8000 and size("kda_pages_compact_workspace_size", -1) == 0
    ws = layers.paged_decode_q8_workspace_size
    assert ws(4, 1000, 8, 2, 128) > 0 and ws(4, 1000, 8, 3, 128) == 0 and ws(0, 1000, 8, 2, 128) == 0
    assert ws(4, 64, 8, 2, 128) == 0 and ws(4, 65, 8, 2, 128) > 0


def test_status_string():
    assert kda.lib().kda_status_string(5).startswith(b"KDA_ERR_NO_PAGES")


def test_binding_refuses_host_tensors():
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = torch.zeros(2, 2, 16, 64, dtype=torch.uint8).view(ref.E4M3)
    s, q = torch.ones(2, 2, 1), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        layers.paged_append_q8(q, q, c, c, s, s, i(3, 2), i(3))
    with pytest.raises(ValueError):
        layers.paged_decode_q8(q, c, c, s, s, i(3, 2), i(3))
    with pytest.raises(ValueError):
        pages.pages_resize(i(3, 2), i(3), i(4), i(3), 16)
    with pytest.raises(ValueError):
        pages.pages_fork([], i(3, 2), i(3), i(4), i(3), i(1), i(1), 16)
    with pytest.raises(ValueError):
        pages.pages_compact([], None, i(4))


def test_plain_rounding():
    """The plain form's rounding is that of torch's type, for all codes and the midpoints between them."""
    codes = torch.arange(256, dtype=torch.uint8).view(ref.E4M3).double()
    codes = codes[torch.isfinite(codes)].unique()
    mid = (codes[1:] + codes[:-1]) / 2
    x = torch.cat([codes, mid, mid * (1 + 1e-6), mid * (1 - 1e-6)]).float()
    assert torch.equal(ref.round_e4m3(x.double()), x.to(ref.E4M3).double())
