"""Cases, plain forms and 64-bit values of the operators around the KDA layers of a hybrid stack.

Five operators, as one serving step of such a stack meets them:

  linear         out = act(x w^T + bias) + residual, the projections before and after a mixer
  decay_prefill  linear attention with one decay per head over packed prompts (chunked form)
  decay_decode   the same mixer for one new token per sequence, states in a pool (recurrent form)
  paged_append   new keys and values written into the pages of a key-value cache
  paged_decode   attention of one new token per sequence over that cache

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true,
through the package's entry points.  ``exact`` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the framework's smallest prompt: 64 float32 tokens, two small heads; all latency
        {"name": "decay prefill, 64 tokens f32", "op": "decay_prefill", "dtype": "f32", "n": 1, "lo": 64, "hi": 64,
         "empty": 0, "H": 2, "dk": 32, "dv": 32, "init": 1, "fused": 0},
        # one 4096-token prompt through a 16-head layer: few chains on many SMs
        {"name": "decay prefill, one prompt", "op": "decay_prefill", "dtype": "bf16", "n": 1, "lo": 4096, "hi": 4096,
         "empty": 0, "H": 16, "dk": 128, "dv": 128, "init": 1, "fused": 0},
        # a packed batch of ragged prompts, one of them empty, q/k/v cut from one fused projection
        {"name": "decay prefill, ragged batch", "op": "decay_prefill", "dtype": "bf16", "n": 64, "lo": 1, "hi": 4096,
         "empty": 1, "H": 32, "dk": 128, "dv": 128, "init": 0, "fused": 1},
        # three live sequences and a padding row in float32: the smallest decode step
        {"name": "decay decode, 4 rows f32", "op": "decay_decode", "dtype": "f32", "n": 4, "pad": 1, "H": 2, "dk": 64,
         "dv": 64, "fused": 0},
        # a full decode batch: 256 sequences, 32 heads, 537 MB of live states
        {"name": "decay decode, 256 rows", "op": "decay_decode", "dtype": "bf16", "n": 256, "pad": 0, "H": 32, "dk": 128,
         "dv": 128, "fused": 1},
        # a decode step: every sequence's new token into its page
        {"name": "paged append, 256 tokens", "op": "paged_append", "dtype": "bf16", "n": 256, "lo": 1, "hi": 1,
         "start": 1000, "H": 8, "d": 128, "ps": 64},
        # prompts of a batch into their pages
        {"name": "paged append, prompts", "op": "paged_append", "dtype": "bf16", "n": 64, "lo": 1, "hi": 4096,
         "start": 100, "H": 8, "d": 128, "ps": 64},
        # a few short float32 sequences, small pages, one of them empty: latency
        {"name": "paged decode, 4 short f32", "op": "paged_decode", "dtype": "f32", "n": 4, "lo": 1, "hi": 50, "empty": 1,
         "Hkv": 2, "G": 2, "d": 64, "ps": 16},
        # one sequence with a long cache: the work of one row spread over the GPU
        {"name": "paged decode, one long row", "op": "paged_decode", "dtype": "bf16", "n": 1, "lo": 131072, "hi": 131072,
         "empty": 0, "Hkv": 8, "G": 4, "d": 128, "ps": 64},
        # a ragged decode batch of a grouped-query layer
        {"name": "paged decode, ragged batch", "op": "paged_decode", "dtype": "bf16", "n": 64, "lo": 1, "hi": 16384,
         "empty": 1, "Hkv": 8, "G": 4, "d": 128, "ps": 64},
        # the output projection of a decode step: few rows, the weights are the traffic
        {"name": "linear, 64 rows", "op": "linear", "m": 64, "n": 4096, "k": 4096, "bias": 1, "act": "none",
         "residual": 1, "out": "bf16"},
        # an input projection over a batch of prompts: all tensor cores
        {"name": "linear, 8192 rows", "op": "linear", "m": 8192, "n": 16384, "k": 4096, "bias": 1, "act": "silu",
         "residual": 0, "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decay_prefill", "decay_prefill", "decay_decode", "paged_append", "paged_decode", "paged_decode",
                     "linear", "linear"])
    dt = "f32" if rng.random() < 0.25 else "bf16"
    if op in ("decay_prefill", "decay_decode"):
        dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (rng.choice([32, 64, 128]), rng.choice([32, 64, 128]))])
        H = _log(rng, 1, 32)
        fused = rng.randrange(2)
        if op == "decay_decode":
            return {"op": op, "dtype": dt, "n": _log(rng, 1, 256), "pad": rng.randrange(3), "H": H, "dk": dk, "dv": dv,
                    "fused": fused}
        n = _log(rng, 1, 64)
        most = (4_000_000 if dt == "bf16" else 250_000) // (n * H)       # tokens per sequence
        hi = _log(rng, 1, max(1, min(65536, most)))
        return {"op": op, "dtype": dt, "n": n, "lo": rng.choice([1, hi]), "hi": hi, "empty": rng.randrange(2) if n > 1 else 0,
                "H": H, "dk": dk, "dv": dv, "init": rng.randrange(2), "fused": fused}
    ps = rng.choice([16, 32, 64, 128])
    Hkv, d = _log(rng, 1, 8), rng.choice([128, 128, 64, 32])
    if op == "paged_append":
        if rng.random() < 0.5:
            return {"op": op, "dtype": dt, "n": _log(rng, 1, 256), "lo": 1, "hi": 1, "start": _log(rng, 1, 2000), "H": Hkv,
                    "d": d, "ps": ps}
        n = _log(rng, 1, 64)
        return {"op": op, "dtype": dt, "n": n, "lo": 1, "hi": _log(rng, 2, 4096 * (1 if dt == "bf16" else 2) // 2),
                "start": _log(rng, 1, 200), "H": Hkv, "d": d, "ps": ps}
    if op == "paged_decode":
        n = _log(rng, 1, 256)
        most = (4_000_000 if dt == "bf16" else 2_000_000) // (n * Hkv)
        hi = _log(rng, 1, max(1, min(131072, most)))
        return {"op": op, "dtype": dt, "n": n, "lo": rng.choice([1, hi]), "hi": hi, "empty": rng.randrange(2) if n > 1 else 0,
                "Hkv": Hkv, "G": rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), "d": d, "ps": ps}
    m, n, k = _log(rng, 1, 8192), _log(rng, 8, 16384), _log(rng, 32, 8192)
    if rng.random() < 0.75:                                              # model widths are mostly multiples of 8
        n, k = -(-n // 8) * 8, -(-k // 8) * 8
    while m * n * k > 500_000_000_000:
        m = max(1, m // 2)
    return {"op": op, "m": m, "n": n, "k": k, "bias": rng.randrange(2), "act": rng.choice(["none", "relu", "gelu", "silu", "sigmoid"]),
            "residual": rng.randrange(2), "out": rng.choice(["bf16", "bf16", "f32"])}


def _lens(c):
    """Lengths spread over [lo, hi] by the case alone (the seed only permutes them)."""
    n, lo, hi = c["n"], c["lo"], c["hi"]
    got = [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) if hi > lo else lo for i in range(n)]
    if c.get("empty"):
        got[0] = 0
    return got


def _starts(c):
    return [int(c["start"] * (((i + 1) * 0.7548776662466927) % 1.0)) for i in range(c["n"])]


def work(case):
    op = case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        o = 2 if case["out"] == "bf16" else 4
        return {"bytes": 2 * (m * k + n * k) + o * m * n * (1 + case["residual"]) + 4 * n * case["bias"], "flops": 2 * m * n * k}
    e = 2 if case["dtype"] == "bf16" else 4
    if op == "decay_prefill":
        T, H, dk, dv, N = sum(_lens(case)), case["H"], case["dk"], case["dv"], case["n"]
        return {"bytes": e * T * H * (2 * dk + 2 * dv) + 4 * N * H * dk * dv * (1 + case["init"]),
                "flops": T * H * 4 * dk * dv}
    if op == "decay_decode":
        live, H, dk, dv = max(0, case["n"] - case["pad"]), case["H"], case["dk"], case["dv"]
        return {"bytes": live * H * (8 * dk * dv + e * (2 * dk + 2 * dv)), "flops": live * H * 5 * dk * dv}
    if op == "paged_append":
        return {"bytes": 4 * e * sum(_lens(case)) * case["H"] * case["d"], "flops": 0}
    T, Hkv, G, d = sum(_lens(case)), case["Hkv"], case["G"], case["d"]
    return {"bytes": e * 2 * T * Hkv * d + case["n"] * Hkv * G * (2 * e * d + 4), "flops": 4 * T * Hkv * G * d}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _perm(x, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return [x[i] for i in torch.randperm(len(x), generator=g).tolist()]


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _qkv(g, T, H, dk, dv, dt, fused):
    """q and k of unit length per head, v normal; with `fused` three slices of one row-major product."""
    def unit(shape):
        x = torch.randn(shape, generator=g, device="cuda")
        return (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)
    q, k = unit((T, H, dk)), unit((T, H, dk))
    v = torch.randn((T, H, dv), generator=g, device="cuda").to(dt)
    if not fused:
        return q, k, v
    a = torch.cat([q.reshape(T, -1), k.reshape(T, -1), v.reshape(T, -1)], dim=1)
    cut = lambda o, d: a[:, o:o + H * d].unflatten(1, (H, d))  # noqa: E731
    return cut(0, dk), cut(H * dk, dk), cut(2 * H * dk, dv)


def _pages(g, lens, ps):
    """A table of randomly placed pages for sequences of these lengths (-1 where there is none)."""
    need = [-(-n // ps) for n in lens]
    total, most = sum(need), max(1, max(need))
    ids = torch.randperm(total + 3, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(most, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[have] = ids
    return table, total + 3


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        ot = DT[case["out"]]
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        return {"case": case, "x": rnd(m, k).to(torch.bfloat16), "w": (rnd(n, k) / math.sqrt(k)).to(torch.bfloat16),
                "bias": 0.1 * rnd(n) if case["bias"] else None, "residual": rnd(m, n).to(ot) if case["residual"] else None}
    dt = DT[case["dtype"]]
    if op in ("decay_prefill", "decay_decode"):
        H, dk, dv, n = case["H"], case["dk"], case["dv"], case["n"]
        lens = _perm(_lens(case), seed) if op == "decay_prefill" else [1] * n
        T = sum(lens)
        q, k, v = _qkv(g, T, H, dk, dv, dt, case["fused"])
        s = {"case": case, "q": q, "k": k, "v": v,
             # per-head rates between 1 and 1/256 a token
             "log_decay": -torch.exp2(-8 * torch.rand(H, generator=g, device="cuda"))}
        if op == "decay_prefill":
            s["cu"] = _i32([0] + torch.tensor(lens).cumsum(0).tolist())
            s["most"] = max(lens)                                        # a scheduler knows it; sizes the plain form's padding
            s["init"] = 0.1 * torch.randn((n, H, dk, dv), generator=g, device="cuda") if case["init"] else None
        else:
            s["pool"] = 0.1 * torch.randn((n + 2, H, dk, dv), generator=g, device="cuda")
            slots = torch.randperm(n + 2, generator=g, device="cuda")[:n].to(torch.int32)
            slots[:min(n, case["pad"])] = -1
            s["slots"] = slots
        return s
    d, ps = case["d"], case["ps"]
    if op == "paged_append":
        H = case["H"]
        both = _perm(list(zip(_lens(case), _starts(case))), seed)
        lens, starts = [x for x, _ in both], [x for _, x in both]
        table, total = _pages(g, [a + b for a, b in both], ps)
        T = sum(lens)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(dt)  # noqa: E731
        one = case["hi"] == 1
        return {"case": case, "k": rnd(T, H, d), "v": rnd(T, H, d), "kc": rnd(total, H, ps, d), "vc": rnd(total, H, ps, d),
                "table": table, "start": _i32(starts), "cu": None if one else _i32([0] + torch.tensor(lens).cumsum(0).tolist())}
    H, G = case["Hkv"], case["G"]
    lens = _perm(_lens(case), seed)
    table, total = _pages(g, lens, ps)
    kc = torch.randn((total, H, ps, d), generator=g, device="cuda", dtype=dt)
    vc = torch.randn((total, H, ps, d), generator=g, device="cuda", dtype=dt)
    # nobody clears a page before use: what no token was written to holds NaN
    pos = torch.arange(table.shape[1] * ps, device="cuda").reshape(1, -1, ps)
    used = pos < torch.tensor(lens, device="cuda")[:, None, None]
    free = torch.ones((total, ps), dtype=torch.bool, device="cuda")
    have = table >= 0
    free[table[have].long()] = ~used[have]
    kc.masked_fill_(free[:, None, :, None], float("nan"))
    vc.masked_fill_(free[:, None, :, None], float("nan"))
    return {"case": case, "q": torch.randn((len(lens), H * G, d), generator=g, device="cuda").to(dt), "kc": kc, "vc": vc,
            "table": table, "lens": _i32(lens), "scale": 1.0 / math.sqrt(d)}


# ---------------------------------------------------------------- plain forms
def _act(y, act):
    if act == "relu":
        return y.clamp(min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "sigmoid":
        return 1 / (1 + torch.exp(-y))
    return y


def _plain_linear(s):
    y = s["x"].float() @ s["w"].float().t()
    if s["bias"] is not None:
        y = y + s["bias"]
    y = _act(y, s["case"]["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(DT[s["case"]["out"]])


def _plain_decay_prefill(s, C=64):
    q, k, v, cu, ld = s["q"], s["k"], s["v"], s["cu"].long(), s["log_decay"]
    N, (T, H, dk), dv = cu.numel() - 1, q.shape, v.shape[2]
    n = max(1, -(-s["most"] // C))
    at = cu[:-1, None] + torch.arange(n * C, device="cuda")              # [N, n C]: padded to whole chunks
    lens = cu[1:] - cu[:-1]
    real = torch.arange(n * C, device="cuda") < lens[:, None]
    at = torch.where(real, at, 0)
    def rows(x):
        if T == 0:
            return torch.zeros((N, n, H, C, x.shape[2]), device="cuda")
        y = torch.where(real[..., None, None], x[at].float(), 0.0)
        return y.unflatten(1, (n, C)).transpose(2, 3)                    # [N, n, H, C, d]
    q, k, v = rows(q), rows(k), rows(v)
    i = torch.arange(C, device="cuda")
    gap = i[:, None] - i[None]
    D = torch.where(gap >= 0, torch.exp(ld[:, None, None] * gap.clamp(min=0)), 0.0)      # [H, C, C]
    out = ((q @ k.transpose(3, 4)) * D) @ v
    # what each chunk adds to the state at its own end, and from there to later chunks
    c0 = torch.arange(n, device="cuda") * C
    end = torch.minimum(c0[None] + C, lens[:, None]).clamp(min=0)                        # [N, n]
    left = (end[..., None] - 1 - c0[None, :, None] - i).clamp(min=0)                     # [N, n, C]
    wk = k * torch.exp(ld[None, None, :, None] * left[:, :, None])[..., None]
    add = wk.transpose(3, 4) @ v                                                         # [N, n, H, dk, dv]
    del wk
    add = add.permute(2, 1, 0, 3, 4).reshape(H, n, -1)
    cgap = c0[:, None] - c0[None] - C
    M = torch.where(cgap >= 0, torch.exp(ld[:, None, None] * cgap.clamp(min=0)), 0.0)    # [H, n, n]
    S = (M @ add).reshape(H, n, N, dk, dv).permute(2, 1, 0, 3, 4)
    init = s["init"]
    if init is not None:
        S = S + torch.exp(ld[:, None] * c0)[None].transpose(1, 2)[..., None, None] * init[:, None]
    out = out + torch.exp(ld[:, None] * (i + 1))[..., None] * (q @ S)
    del S
    out = out.transpose(2, 3).flatten(1, 2)[real].to(s["q"].dtype)
    rest = torch.where(end > c0, lens[:, None] - end, -1)
    wf = torch.where((rest >= 0)[..., None], torch.exp(rest.clamp(min=0)[..., None] * ld), 0.0)   # [N, n, H]
    final = torch.einsum("nch,hcnx->nhx", wf, add.reshape(H, n, N, dk * dv)).reshape(N, H, dk, dv)
    if init is not None:
        final = final + torch.exp(lens[:, None] * ld)[..., None, None] * init
    return out, final


def _plain_decay_decode(s):
    q, k, v, slots, pool = s["q"].float(), s["k"].float(), s["v"].float(), s["slots"].long(), s["pool"]
    live = slots >= 0
    S = pool[slots.clamp(min=0)] * torch.exp(s["log_decay"])[:, None, None] + k[..., None] * v[..., None, :]
    out = torch.where(live[:, None, None], (q[..., None] * S).sum(2), 0.0).to(s["q"].dtype)
    pool[slots[live]] = S[live]
    return out, pool


def _plain_paged_append(s):
    k, v, kc, vc, table, start = s["k"], s["v"], s["kc"], s["vc"], s["table"].long(), s["start"].long()
    T, H, ps = k.shape[0], k.shape[1], kc.shape[2]
    t = torch.arange(T, device="cuda")
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(start.numel() + 1, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = start[seq] + t - cu[seq]
    page = table[seq, pos // ps]
    h = torch.arange(H, device="cuda")
    kc[page[:, None], h[None], (pos % ps)[:, None]] = k
    vc[page[:, None], h[None], (pos % ps)[:, None]] = v
    return kc, vc


def _plain_paged_decode(s):
    q, kc, vc, table, lens = s["q"].float(), s["kc"], s["vc"], s["table"].long(), s["lens"].long()
    N, Hq, d = q.shape
    Hkv, ps = kc.shape[1], kc.shape[2]
    pos = torch.arange(table.shape[1] * ps, device="cuda")
    real = pos[None] < lens[:, None]                                     # [N, L]
    at = table.clamp(min=0)
    def rows(c):
        x = c[at].transpose(1, 2).flatten(2, 3)                          # [N, Hkv, L, d]
        return torch.where(real[:, None, :, None], x.float(), 0.0)
    sc = (q.reshape(N, Hkv, Hq // Hkv, d) @ rows(kc).transpose(2, 3)) * s["scale"]
    sc = torch.where(real[:, None, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m0)
    l = p.sum(-1, keepdim=True)
    out = (p @ rows(vc)) / torch.where(l == 0, 1.0, l)
    return out.reshape(N, Hq, d).to(s["q"].dtype), (m0 + torch.log(l)).reshape(N, Hq)


_PLAIN = {"linear": _plain_linear, "decay_prefill": _plain_decay_prefill, "decay_decode": _plain_decay_decode,
          "paged_append": _plain_paged_append, "paged_decode": _plain_paged_decode}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    import gated_delta_rule_46_gb300 as pkg
    if op == "linear":
        return pkg.linear(s["x"], s["w"], bias=s["bias"], residual=s["residual"], act=s["case"]["act"],
                          out_dtype=DT[s["case"]["out"]])
    if op == "decay_prefill":
        return pkg.decay_prefill(s["q"], s["k"], s["v"], s["log_decay"], s["cu"], initial_state=s["init"])
    if op == "decay_decode":
        return pkg.decay_decode(s["q"], s["k"], s["v"], s["log_decay"], s["pool"], slot_ids=s["slots"]), s["pool"]
    if op == "paged_append":
        pkg.paged_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["start"], cu_seqlens=s["cu"])
        return s["kc"], s["vc"]
    return pkg.paged_decode(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"], return_lse=True)


# ---------------------------------------------------------------- 64-bit values
def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "linear":
        y = torch.matmul(s["x"].double(), s["w"].double().t())
        if s["bias"] is not None:
            y += s["bias"].double()
        a = case["act"]
        if a == "relu":
            y = torch.maximum(y, torch.zeros_like(y))
        elif a == "gelu":
            y = y * 0.5 * torch.special.erfc(-y / math.sqrt(2.0))
        elif a == "silu":
            y = y * torch.special.expit(y)
        elif a == "sigmoid":
            y = torch.special.expit(y)
        if s["residual"] is not None:
            y += s["residual"].double()
        return y
    if op == "decay_prefill":
        # the recurrence token by token, the sequences that still have tokens side by side
        cu = s["cu"].tolist()
        lens = [b - a for a, b in zip(cu, cu[1:])]
        order = sorted(range(len(lens)), key=lambda i: -lens[i])
        N, H, dk, dv = len(lens), case["H"], case["dk"], case["dv"]
        at = torch.tensor(order, device="cuda")
        first = s["cu"][:-1].long()[at]
        lam = s["log_decay"].double().exp()[:, None, None]
        S = torch.zeros((N, H, dk, dv), dtype=torch.float64, device="cuda")
        if s["init"] is not None:
            S += s["init"].double()[at]
        out = torch.zeros((cu[-1], H, dv), dtype=torch.float64, device="cuda")
        alive = N
        for t in range(max(lens)):
            while lens[order[alive - 1]] <= t:
                alive -= 1
            r = first[:alive] + t
            A = S[:alive]
            A.mul_(lam).add_(s["k"][r].double()[..., None] * s["v"][r].double()[..., None, :])
            out[r] = torch.matmul(s["q"][r].double()[..., None, :], A)[..., 0, :]
        final = torch.empty_like(S)
        final[at] = S
        return out, final
    if op == "decay_decode":
        pool = s["pool"].double()
        out = torch.zeros((case["n"], case["H"], case["dv"]), dtype=torch.float64, device="cuda")
        lam = s["log_decay"].double().exp()[:, None, None]
        for i, slot in enumerate(s["slots"].tolist()):
            if slot >= 0:
                pool[slot] = lam * pool[slot] + torch.einsum("hk,hv->hkv", s["k"][i].double(), s["v"][i].double())
                out[i] = torch.einsum("hk,hkv->hv", s["q"][i].double(), pool[slot])
        return out, pool
    table = s["table"].tolist()
    if op == "paged_append":
        kc, vc, ps = s["kc"].double(), s["vc"].double(), case["ps"]
        starts = s["start"].tolist()
        cu = s["cu"].tolist() if s["cu"] is not None else list(range(case["n"] + 1))
        for i, p0 in enumerate(starts):
            t, p = cu[i], p0
            while t < cu[i + 1]:                                         # page by page
                m = min(ps - p % ps, cu[i + 1] - t)
                for c, x in ((kc, s["k"]), (vc, s["v"])):
                    c[table[i][p // ps], :, p % ps:p % ps + m] = x[t:t + m].transpose(0, 1).double()
                t, p = t + m, p + m
        return kc, vc
    q, ps, H, G, d = s["q"].double(), case["ps"], case["Hkv"], case["G"], case["d"]
    out = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        ids = s["table"][i, :-(-n // ps)].long()
        K, V = (c[ids].permute(1, 0, 2, 3).reshape(H, -1, d)[:, :n].double() for c in (s["kc"], s["vc"]))
        sc = torch.einsum("hgd,hnd->hgn", q[i].reshape(H, G, d), K) * s["scale"]
        z = torch.logsumexp(sc, -1)
        out[i] = torch.einsum("hgn,hnd->hgd", torch.exp(sc - z[..., None]), V).reshape(H * G, d)
        lse[i] = z.reshape(-1)
    return out, lse
