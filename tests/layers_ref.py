"""Plain 64-bit forms of the layer operators, from their definitions, on the CPU.

Tolerances (rel-L2 = ||x - y|| / ||y||), fixed here for every test of these
operators.  A float32 result is a sum of up to a few thousand rounded terms: its
rounding errors, 2^-24 of a term each and of either sign, stay far below 1e-5 of
the result.  A bf16 result is rounded once, by at most 2^-9 of itself; where its
operator also rounds an intermediate factor to bf16 for the tensor cores (the
softmax weights; the state and the decayed products of linear attention), each
such rounding moves a term of the sum by at most 2^-9 of itself: 3 * 2^-9 in all.
"""
import math

import torch

F32_TOL = 1e-5
BF16_TOL = 3 * 2.0 ** -9


def tol(dtype):
    return BF16_TOL if dtype == torch.bfloat16 else F32_TOL


def rel(got, ref):
    g, r = got.detach().double().cpu(), ref.double().cpu()
    assert g.shape == r.shape, (g.shape, r.shape)
    assert torch.equal(torch.isfinite(g), torch.isfinite(r)), "finite in other places"
    assert torch.equal(torch.isnan(g), torch.isnan(r)), "NaN in other places"
    inf = torch.isinf(r)
    assert torch.equal(g[inf], r[inf]), "another infinity"
    fine = torch.isfinite(r)
    d, n = (g - r)[fine].norm(), r[fine].norm()
    return float(d / n) if n > 0 else float(d)


def close(name, got, ref, dtype=None):
    e, t = rel(got, ref), tol(dtype or got.dtype)
    assert e <= t, f"{name}: rel-L2 {e:.3e} > {t:.3e}"


def linear(x, w, bias, residual, act):
    y = x.double() @ w.double().t()
    if bias is not None:
        y = y + bias.double()
    y = {"none": lambda a: a, "relu": torch.relu, "silu": lambda a: a * torch.sigmoid(a), "sigmoid": torch.sigmoid,
         "gelu": lambda a: a * 0.5 * torch.special.erfc(-a / math.sqrt(2.0))}[act](y)
    return y if residual is None else y + residual.double()


def decay(q, k, v, log_decay, lens, init=None, scale=1.0):
    """Token by token.  q, k [T, H, dk], v [T, H, dv]; returns out [T, H, dv], final [N, H, dk, dv]."""
    T, H, dk = q.shape
    dv = v.shape[2]
    lam = torch.exp(log_decay.double())[:, None, None]
    out, fin, t = torch.zeros(T, H, dv, dtype=torch.float64), [], 0
    for i, n in enumerate(lens):
        S = torch.zeros(H, dk, dv, dtype=torch.float64) if init is None else init[i].double().clone()
        for _ in range(n):
            S = lam * S + k[t].double()[:, :, None] * v[t].double()[:, None, :]
            out[t] = scale * torch.einsum("hk,hkv->hv", q[t].double(), S)
            t += 1
        fin.append(S)
    return out, torch.stack(fin)


def paged(q, kc, vc, table, lens, scale):
    """q [N, Hq, d], caches [P, Hkv, ps, d]; tokens on pages outside the cache are left out."""
    N, Hq, d = q.shape
    P, Hkv, ps, _ = kc.shape
    out = torch.zeros(N, Hq, d, dtype=torch.float64)
    lse = torch.full((N, Hq), -math.inf, dtype=torch.float64)
    for i, n in enumerate(lens):
        at = [(int(table[i, t // ps]), t % ps) for t in range(n)]
        at = [(p, o) for p, o in at if 0 <= p < P]
        if not at:
            continue
        p, o = torch.tensor([a for a, _ in at]), torch.tensor([b for _, b in at])
        K, V = kc[p, :, o].double(), vc[p, :, o].double()               # [n, Hkv, d]
        for h in range(Hq):
            s = scale * (K[:, h // (Hq // Hkv)] @ q[i, h].double())
            lse[i, h] = torch.logsumexp(s, 0)
            out[i, h] = torch.softmax(s, 0) @ V[:, h // (Hq // Hkv)]
    return out, lse


def fused_rows(parts, dev):
    """The tensors [T, H, d_i] as slices of one [T, sum H d_i + 8] product (rows 16 bytes apart from dense)."""
    T = parts[0].shape[0]
    flat = torch.cat([p.reshape(T, -1) for p in parts] + [torch.zeros(T, 8, dtype=parts[0].dtype)], 1).to(dev)
    got, at = [], 0
    for p in parts:
        n = p.shape[1] * p.shape[2]
        got.append(flat[:, at:at + n].unflatten(1, p.shape[1:]))
        at += n
    return got
