"""Cases, plain forms and 64-bit values of the operators of a key-value cache in 8 bits and of its pages.

Five operators, as the full-attention layers of a served hybrid stack meet them:

  append    new keys and values into an e4m3 cache with a power-of-two scale for each block of tokens and head
  decode    attention of one new token per sequence over that cache
  resize    pages given to rows of the page table that grow, and taken back from rows that shrink or end
  fork      rows that go on from another row's tokens: full pages shared, the last one copied in all pools
  compact   pages in use moved to the front of all pools

``run`` computes them with elementary torch operations, or, where ``own`` is true, through the
package's entry points.  ``exact`` computes them from their definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
E4M3 = torch.float8_e4m3fn


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a decode step: every sequence's new token into its page
        {"name": "append, 256 tokens", "op": "append", "dtype": "bf16", "n": 256, "lo": 1, "hi": 1, "start": 1000, "H": 8,
         "d": 128, "ps": 64, "block": 16},
        # prompts of a batch into their pages, from positions inside blocks on (their earlier parts were cached before)
        {"name": "append, prompts", "op": "append", "dtype": "bf16", "n": 64, "lo": 1, "hi": 4096, "start": 100, "H": 8,
         "d": 128, "ps": 64, "block": 16},
        # a few short float32 sequences, small pages, one of them empty: latency
        {"name": "decode, 4 short f32", "op": "decode", "dtype": "f32", "n": 4, "lo": 1, "hi": 50, "empty": 1, "Hkv": 2, "G": 2,
         "d": 64, "ps": 16, "block": 16},
        # one sequence with a long cache: the work of one row spread over the GPU
        {"name": "decode, one long row", "op": "decode", "dtype": "bf16", "n": 1, "lo": 131072, "hi": 131072, "empty": 0,
         "Hkv": 8, "G": 4, "d": 128, "ps": 64, "block": 16},
        # a ragged decode batch of a grouped-query layer
        {"name": "decode, ragged batch", "op": "decode", "dtype": "bf16", "n": 64, "lo": 1, "hi": 16384, "empty": 1, "Hkv": 8,
         "G": 4, "d": 128, "ps": 64, "block": 16},
        # many query heads to a key-value head of 64 channels, long blocks
        {"name": "decode, 16 heads share 64 ch", "op": "decode", "dtype": "bf16", "n": 128, "lo": 1, "hi": 8192, "empty": 0,
         "Hkv": 4, "G": 16, "d": 64, "ps": 32, "block": 32},
        # a step of speculative decoding: drafts cut back to what was accepted, room for the next draft
        {"name": "resize, drafts of 256 rows", "op": "resize", "n": 256, "lo": 1, "hi": 8192, "low": "draft", "ps": 64,
         "spare": 4096},
        # a large batch turned over: rows that ended give their pages back, as many prompts get theirs
        {"name": "resize, 512 rows turned over", "op": "resize", "n": 512, "lo": 1, "hi": 32768, "low": "half", "ps": 64,
         "spare": 16384},
        # four beams of one short prompt, a small float32-scaled cache of two layers
        {"name": "fork, 4 beams", "op": "fork", "n": 8, "lo": 20, "hi": 60, "forks": 4, "ps": 16, "H": 2, "d": 64, "block": 16,
         "layers": 2},
        # samples of many prompts, all layers' pools
        {"name": "fork, 192 rows", "op": "fork", "n": 400, "lo": 1, "hi": 600, "forks": 192, "ps": 64, "H": 8, "d": 128,
         "block": 16, "layers": 12},
        # a small pool with a few holes
        {"name": "compact, few pages", "op": "compact", "n": 16, "lo": 1, "hi": 200, "gone": 25, "ps": 16, "H": 2, "d": 64,
         "block": 16, "layers": 2},
        # half of a batch has ended: what is left moves to the front
        {"name": "compact, half of a batch gone", "op": "compact", "n": 128, "lo": 1, "hi": 2048, "gone": 50, "ps": 64, "H": 8,
         "d": 128, "block": 16, "layers": 12},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "decode", "decode", "decode", "resize", "fork", "compact"])
    ps = rng.choice([16, 32, 64, 128])
    block = rng.choice([b for b in (16, 16, 32, 64, 128) if b <= ps])
    H, d = _log(rng, 1, 8), rng.choice([128, 128, 64, 32])
    dt = "f32" if rng.random() < 0.25 else "bf16"
    if op == "append":
        c = {"op": op, "dtype": dt, "H": H, "d": d, "ps": ps, "block": block}
        if rng.random() < 0.5:
            return {**c, "n": _log(rng, 1, 256), "lo": 1, "hi": 1, "start": _log(rng, 1, 2000)}
        return {**c, "n": _log(rng, 1, 64), "lo": 1, "hi": _log(rng, 2, 4096 if dt == "bf16" else 2048), "start": _log(rng, 1, 200)}
    if op == "decode":
        n = _log(rng, 1, 256)
        hi = _log(rng, 1, max(1, min(131072, (4_000_000 if dt == "bf16" else 1_000_000) // (n * H))))
        return {"op": op, "dtype": dt, "n": n, "lo": rng.choice([1, hi]), "hi": hi, "empty": rng.randrange(2) if n > 1 else 0,
                "Hkv": H, "G": rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), "d": d, "ps": ps, "block": block}
    if op == "resize":
        return {"op": op, "n": _log(rng, 1, 512), "lo": 1, "hi": _log(rng, 2, 32768), "low": rng.choice(["draft", "half"]),
                "ps": ps, "spare": _log(rng, 16, 16384)}
    c = {"op": op, "lo": 1, "hi": _log(rng, 20, 1000), "ps": ps, "H": H, "d": d, "block": block, "layers": _log(rng, 1, 12)}
    if op == "fork":
        forks = _log(rng, 1, 128)
        return {**c, "n": forks + _log(rng, 1, 64), "forks": forks}
    return {**c, "n": _log(rng, 2, 128), "gone": rng.choice([10, 25, 50, 75])}


def _lens(c):
    """Lengths spread over [lo, hi] by the case alone (the seed only permutes them)."""
    n, lo, hi = c["n"], c["lo"], c["hi"]
    got = [lo + int((hi - lo + 1) * (((i + 1) * 0.6180339887498949) % 1.0)) if hi > lo else lo for i in range(n)]
    if c.get("empty"):
        got[0] = 0
    return got


def _starts(c):
    return [int(c["start"] * (((i + 1) * 0.7548776662466927) % 1.0)) for i in range(c["n"])]


def _up(n, m):
    return -(-n // m)


def _low_high(c):
    """resize: the tokens that each row is cut back to (-1: as it is), and those that it then has room for."""
    high = _lens(c)
    if c["low"] == "draft":                                              # eight drafted tokens, some of them accepted
        return [max(0, n - 1 - (i * 5) % 8) for i, n in enumerate(high)], high
    return [0 if i % 2 else -1 for i in range(len(high))], high


def _page_bytes(c):
    """Bytes of one page in all pools of a layer: e4m3 keys and values, float32 scales."""
    return 2 * c["H"] * (c["ps"] * c["d"] + 4 * (c["ps"] // c["block"]))


def work(case):
    op = case["op"]
    if op == "append":
        e, T, H, d, B = 2 if case["dtype"] == "bf16" else 4, sum(_lens(case)), case["H"], case["d"], case["block"]
        blocks = sum(_up(s % B + n, B) for s, n in zip(_starts(case), _lens(case)))
        return {"bytes": 2 * T * H * d * (e + 1) + 2 * 4 * blocks * H, "flops": 4 * T * H * d}
    if op == "decode":
        e, T, Hkv, G, d = 2 if case["dtype"] == "bf16" else 4, sum(_lens(case)), case["Hkv"], case["G"], case["d"]
        blocks = sum(_up(n, case["block"]) for n in _lens(case))
        return {"bytes": 2 * T * Hkv * d + 8 * blocks * Hkv + case["n"] * Hkv * G * (2 * e * d + 4), "flops": 4 * T * Hkv * G * d}
    ps, n = case["ps"], case["n"]
    if op == "resize":
        low, high = _low_high(case)
        moved = sum(_up(b, ps) - _up(a, ps) for a, b in zip(low, high) if a >= 0)
        # tokens and pages held, twice; of a page given back or out: its table entry and its count, read or written
        return {"bytes": 2 * 12 * n + 2 * 12 * moved, "flops": 0}
    if op == "fork":
        part = [_lens(case)[s] for s in _fork_rows(case)[0]]
        full = sum(p // ps for p in part)
        return {"bytes": 2 * case["layers"] * _page_bytes(case) * sum(p % ps > 0 for p in part) + 12 * full, "flops": 0}
    pages, live, moved = _compaction(case)
    return {"bytes": 2 * case["layers"] * _page_bytes(case) * moved + 8 * live + 8 * pages, "flops": 0}


def _fork_rows(c):
    """Rows that are gone on from, and the rows that do: the last `forks` rows of the table, of the others in turn."""
    first = c["n"] - c["forks"]
    return [i % first for i in range(c["forks"])], list(range(first, c["n"]))


def _gone(c):
    return [(i * 37) % 100 < c["gone"] for i in range(c["n"])]


def _compaction(c):
    """Pages in all, pages in use, and pages that move, where pages were handed out row by row."""
    use = []
    for n, g in zip(_lens(c), _gone(c)):
        use += [not g] * _up(n, c["ps"])
    live = sum(use)
    return len(use), live, sum(use[live:])


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


def _pages(g, lens, ps, spare=3, most=None):
    """A table of randomly placed pages for sequences of these lengths (-1 where there is none)."""
    need = [_up(n, ps) for n in lens]
    total, most = sum(need), max(1, max(need)) if most is None else most
    ids = torch.randperm(total + spare, generator=g, device="cuda")[:total].to(torch.int32)
    table = torch.full((len(lens), most), -1, dtype=torch.int32, device="cuda")
    have = torch.arange(most, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[have] = ids
    return table, total + spare


def _quantised(g, P, H, ps, d, B):
    """A cache's codes and scales as an append leaves them: values of different size from block to block."""
    x = torch.randn((P, H, ps // B, B * d), generator=g, device="cuda")
    x *= torch.exp(torch.randn((P, H, ps // B, 1), generator=g, device="cuda"))
    m, e = torch.frexp(x.abs().amax(-1) / 448)
    scale = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e))
    return (x / scale[..., None]).to(E4M3).reshape(P, H, ps, d), scale


def _pools(g, c, P):
    """Keys, values and their scales of all layers: any bytes will do for what only moves them."""
    H, ps, d, B = c["H"], c["ps"], c["d"], c["block"]
    kv = lambda: torch.randint(0, 0x78, (P, H, ps, d), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)  # noqa: E731
    sc = lambda: torch.rand((P, H, ps // B), generator=g, device="cuda")  # noqa: E731
    return [f() for _ in range(c["layers"]) for f in (kv, kv, sc, sc)]


def _refs(table, P):
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    ids = table[table >= 0].long()
    return refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))


def prepare(case, seed):
    g, op, ps = _gen(seed), case["op"], case["ps"]
    if op == "append":
        dt, H, d, B = DT[case["dtype"]], case["H"], case["d"], case["block"]
        both = _perm(list(zip(_lens(case), _starts(case))), seed)
        lens, starts = [x for x, _ in both], [x for _, x in both]
        table, total = _pages(g, [a + b for a, b in both], ps)
        T = sum(lens)
        # channels of different size, and some tokens whose block's scale grows
        size = torch.exp(0.5 * torch.randn((1, H, d), generator=g, device="cuda"))
        rnd = lambda: (torch.randn((T, H, d), generator=g, device="cuda") * size).to(dt)  # noqa: E731
        k, v = rnd(), rnd()
        (kc, ks), (vc, vs) = _quantised(g, total, H, ps, d, B), _quantised(g, total, H, ps, d, B)
        one = case["hi"] == 1
        return {"case": case, "k": k, "v": v, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table, "start": _i32(starts),
                "cu": None if one else _i32([0] + torch.tensor(lens).cumsum(0).tolist())}
    if op == "decode":
        dt, H, G, d, B = DT[case["dtype"]], case["Hkv"], case["G"], case["d"], case["block"]
        lens = _perm(_lens(case), seed)
        table, total = _pages(g, lens, ps)
        (kc, ks), (vc, vs) = _quantised(g, total, H, ps, d, B), _quantised(g, total, H, ps, d, B)
        # nobody clears a page before use: codes that no token was written to are NaN, and so are their blocks' scales
        pos = torch.arange(table.shape[1] * ps, device="cuda").reshape(1, -1, ps)
        used = pos < torch.tensor(lens, device="cuda")[:, None, None]
        free = torch.ones((total, ps), dtype=torch.bool, device="cuda")
        have = table >= 0
        free[table[have].long()] = ~used[have]
        for c, s in ((kc, ks), (vc, vs)):
            c.view(torch.uint8).masked_fill_(free[:, None, :, None], 0x7F)
            s.masked_fill_(free.unflatten(1, (-1, B)).all(-1)[:, None], math.nan)
        q = torch.randn((len(lens), H * G, d), generator=g, device="cuda").to(dt)
        return {"case": case, "q": q, "kc": kc, "vc": vc, "ks": ks, "vs": vs, "table": table, "lens": _i32(lens),
                "scale": 0.5 / math.sqrt(d)}
    if op == "resize":
        low, high = _low_high(case)
        both = _perm(list(zip(low, high)), seed)
        low, high = [a for a, _ in both], [b for _, b in both]
        table, P = _pages(g, high, ps, spare=case["spare"], most=_up(case["hi"], ps) + 4)
        # some first pages are another row's too (a common prefix)
        table[1::4, 0] = table[0::4, 0][: table[1::4].shape[0]]
        return {"case": case, "table": table, "held": _i32([_up(n, ps) for n in high]), "refs": _refs(table, P),
                "low": _i32(low), "high": _i32(high)}
    lens = _perm(_lens(case), seed) if op == "compact" else _lens(case)
    if op == "fork":
        src, dst = _fork_rows(case)
        for i in dst:
            lens[i] = 0
        table, P = _pages(g, lens, ps, spare=case["forks"] + 5, most=_up(case["hi"], ps) + 1)
        none = [-1] * case["n"]
        for i in dst:
            none[i] = 0
        return {"case": case, "pools": _pools(g, case, P), "table": table, "held": _i32([_up(n, ps) for n in lens]),
                "refs": _refs(table, P), "lens": _i32(lens), "src": _i32(src), "dst": _i32(dst), "losers": _i32(none)}
    # pages handed out in the rows' order, those of ended rows given back
    need = torch.tensor([_up(n, ps) for n in lens], device="cuda")
    P, most = int(need.sum()), int(need.max())
    have = torch.arange(most, device="cuda")[None] < need[:, None]
    table = torch.full((case["n"], most), -1, dtype=torch.int32, device="cuda")
    table[have] = torch.arange(P, dtype=torch.int32, device="cuda")
    gone = torch.tensor(_perm(_gone(case), seed), device="cuda")         # the same order as the lengths'
    table[gone] = -1
    return {"case": case, "pools": _pools(g, case, P), "table": table, "refs": _refs(table, P), "table0": table.clone(),
            "refs0": _refs(table, P)}


# ---------------------------------------------------------------- plain forms
def _put8(x, code, scale, page, at, seq, pos, start, table, live):
    """x [T, H, d] into codes [P, H, ps, d] and scales [P, H, ps / B]; a token's page, place, sequence and position."""
    P, H, ps, d = code.shape
    B = ps // scale.shape[2]
    per, u8 = ps // B, code.view(torch.uint8)
    x = x.float()
    a = x.abs()
    a = torch.where(a < math.inf, a, 0.0).amax(-1)                       # [T, H]; neither infinities nor NaN
    blk = page * per + at // B
    amax = torch.zeros((P * per, H), device="cuda").scatter_reduce_(0, blk[:, None].expand(-1, H), a, "amax")
    hit = torch.zeros(P * per, dtype=torch.bool, device="cuda").index_fill_(0, blk, True)
    m, e = torch.frexp(amax.double() / 448)
    need = torch.ldexp(torch.ones_like(m), torch.where(m == 0.5, e - 1, e).clamp(min=-126)).float()
    flat = scale.transpose(1, 2).reshape(P * per, H)
    # blocks that hold earlier tokens: their scale can only grow, and these tokens follow it
    row = torch.arange(start.numel(), device="cuda")
    inside = start[live] % B
    part = table[row[live], start[live] // ps] * per + start[live] % ps // B
    part, inside = part[inside > 0], inside[inside > 0]
    was = flat[part]
    need[part] = torch.maximum(need[part], was)
    now = torch.where(hit[:, None], need, flat)
    r = torch.arange(B, device="cuda")
    pp, r0 = part // per, part % per * B
    i = (pp[:, None, None], torch.arange(H, device="cuda")[None, :, None], (r0[:, None] + r)[:, None])
    old = u8[i]                                                          # [parts, H, B, d]
    new = (old.view(E4M3).float() * (was / now[part])[..., None, None]).to(E4M3).view(torch.uint8)
    u8[i] = torch.where((r < inside[:, None])[:, None, :, None], new, old)
    y = (x / now[blk][..., None]).to(E4M3).view(torch.uint8)
    u8[page[:, None], torch.arange(H, device="cuda")[None], at[:, None]] = y
    scale.copy_(now.reshape(P, per, H).transpose(1, 2))


def _plain_append(s):
    k, v, table, start, ps = s["k"], s["v"], s["table"].long(), s["start"].long(), s["kc"].shape[2]
    t = torch.arange(k.shape[0], device="cuda")
    cu = s["cu"].long() if s["cu"] is not None else torch.arange(start.numel() + 1, device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    pos = start[seq] + t - cu[seq]
    page = table[seq, pos // ps]
    live = cu[1:] > cu[:-1]
    _put8(k, s["kc"], s["ks"], page, pos % ps, seq, pos, start, table, live)
    _put8(v, s["vc"], s["vs"], page, pos % ps, seq, pos, start, table, live)
    return s["kc"], s["vc"], s["ks"], s["vs"]


def _plain_decode(s):
    q, table, lens = s["q"].float(), s["table"].long(), s["lens"].long()
    N, Hq, d = q.shape
    Hkv, ps = s["kc"].shape[1], s["kc"].shape[2]
    B = ps // s["ks"].shape[2]
    real = torch.arange(table.shape[1] * ps, device="cuda")[None] < lens[:, None]        # [N, L]
    at = table.clamp(min=0)
    def rows(c, scale):
        x = c.view(torch.uint8)[at].view(E4M3).float() * scale[at].repeat_interleave(B, -1)[..., None]
        return x.transpose(1, 2).flatten(2, 3).masked_fill_(~real[:, None, :, None], 0.0)  # [N, Hkv, L, d]
    sc = (q.reshape(N, Hkv, Hq // Hkv, d) @ rows(s["kc"], s["ks"]).transpose(2, 3)) * s["scale"]
    sc = torch.where(real[:, None, None], sc, -math.inf)
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(sc - m0)
    l = p.sum(-1, keepdim=True)
    out = (p @ rows(s["vc"], s["vs"])) / torch.where(l == 0, 1.0, l)
    return out.reshape(N, Hq, d).to(s["q"].dtype), (m0 + torch.log(l)).reshape(N, Hq)


def _plain_resize_one(table, held, refs, tokens, ps):
    col = torch.arange(table.shape[1], device="cuda")[None]
    want = torch.where(tokens < 0, held, (tokens + ps - 1) // ps)
    back = (col >= want[:, None]) & (col < held[:, None])
    ids = table[back].long()
    refs.index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    table.masked_fill_(back, -1)
    get = (col >= held[:, None]) & (col < want[:, None])
    rank = (get.reshape(-1).cumsum(0) - 1).reshape(get.shape)
    free = torch.nonzero(refs == 0)[:, 0]
    get &= rank < free.numel()
    page = free[rank[get]]
    table[get] = page.to(torch.int32)
    refs[page] = 1
    held.copy_(torch.minimum(held, want) + get.sum(1))


def _plain_resize(s):
    _plain_resize_one(s["table"], s["held"], s["refs"], s["low"], s["case"]["ps"])
    _plain_resize_one(s["table"], s["held"], s["refs"], s["high"], s["case"]["ps"])
    return s["table"], s["held"], s["refs"]


def _copy_pages(x, src, dst):
    x = x.view(torch.uint8) if x.dtype == E4M3 else x
    x[dst] = x[src]
    return x


def _plain_fork(s):
    table, held, refs, lens, ps = s["table"], s["held"], s["refs"], s["lens"], s["case"]["ps"]
    _plain_resize_one(table, held, refs, s["losers"], ps)
    src, dst = s["src"].long(), s["dst"].long()
    n = lens[src].long()
    full, part = n // ps, n % ps > 0
    free = torch.nonzero(refs == 0)[:, 0]
    new = free[(part.cumsum(0) - 1)[part]]
    old = table[src[part], full[part]].long()
    share = torch.arange(table.shape[1], device="cuda")[None] < full[:, None]
    rows = torch.where(share, table[src], -1)
    ids = rows[share].long()
    refs.index_add_(0, ids, torch.ones_like(ids, dtype=torch.int32))
    rows[part, full[part]] = new.to(torch.int32)
    refs[new] = 1
    table[dst] = rows
    held[dst] = ((n + ps - 1) // ps).to(torch.int32)
    lens[dst] = n.to(torch.int32)
    [_copy_pages(x, old, new) for x in s["pools"]]
    return s["pools"], table, held, refs, lens


def _plain_compact(s):
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"])                                             # the scheduler's own, as it stands before the call
    refs.copy_(s["refs0"])
    P = refs.numel()
    use = refs != 0
    live = use.sum()
    at = torch.arange(P, device="cuda")
    hole, mover = torch.nonzero(~use & (at < live))[:, 0], torch.nonzero(use & (at >= live))[:, 0]
    to = torch.where(use, at, -1)
    to[mover] = hole
    [_copy_pages(x, mover, hole) for x in s["pools"]]
    refs[hole] = refs[mover]
    refs[mover] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    return s["pools"], table, refs, to.to(torch.int32), live.to(torch.int32).reshape(1)


_PLAIN = {"append": _plain_append, "decode": _plain_decode, "resize": _plain_resize, "fork": _plain_fork,
          "compact": _plain_compact}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return _PLAIN[op](s)
    import gated_delta_rule_46_gb300 as pkg
    if op == "append":
        pkg.paged_append_q8(s["k"], s["v"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["start"], cu_seqlens=s["cu"])
        return s["kc"], s["vc"], s["ks"], s["vs"]
    if op == "decode":
        return pkg.paged_decode_q8(s["q"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["lens"], scale=s["scale"],
                                   return_lse=True)
    if op == "resize":
        pkg.pages_resize(s["table"], s["held"], s["refs"], s["low"], s["case"]["ps"])
        pkg.pages_resize(s["table"], s["held"], s["refs"], s["high"], s["case"]["ps"])
        return s["table"], s["held"], s["refs"]
    if op == "fork":
        pkg.pages_resize(s["table"], s["held"], s["refs"], s["losers"], s["case"]["ps"])
        pkg.pages_fork(s["pools"], s["table"], s["held"], s["refs"], s["lens"], s["src"], s["dst"], s["case"]["ps"])
        return s["pools"], s["table"], s["held"], s["refs"], s["lens"]
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    page_map, live = pkg.pages_compact(s["pools"], s["table"], s["refs"])
    return s["pools"], s["table"], s["refs"], page_map, live


# ---------------------------------------------------------------- 64-bit values
def _e4m3(y):
    """The nearest value with four significant bits and no exponent below -6, ties to the even one."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step


def exact(case, seed):
    s, op, ps = prepare(case, seed), case["op"], case["ps"]
    if op == "append":
        B, table = case["block"], s["table"].tolist()
        starts = s["start"].tolist()
        cu = s["cu"].tolist() if s["cu"] is not None else list(range(case["n"] + 1))
        out = []
        for x, c, scale in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
            c, scale = c.double(), scale.double()
            for i, p0 in enumerate(starts):
                t, p = cu[i], p0
                while t < cu[i + 1]:                                     # block by block
                    m, r, page = min(B - p % B, cu[i + 1] - t), p % B, table[i][p // ps]
                    b = p % ps // B
                    y = x[t:t + m].transpose(0, 1).double()              # [H, m, d]
                    big = y.abs().amax((1, 2)) / 448
                    e = torch.ceil(torch.log2(big)).clamp(min=-126)
                    e = torch.where(torch.exp2(e) < big, e + 1, torch.where(torch.exp2(e - 1) >= big, e - 1, e))
                    f = torch.exp2(e)
                    if r:
                        f = torch.maximum(f, scale[page, :, b])
                        ratio = (scale[page, :, b] / f)[:, None, None]
                        c[page, :, b * B:b * B + r] = _e4m3(c[page, :, b * B:b * B + r] * ratio)
                    scale[page, :, b] = f
                    c[page, :, b * B + r:b * B + r + m] = _e4m3(y / f[:, None, None])
                    t, p = t + m, p + m
            out.append((c, scale))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    if op == "decode":
        q, B, H, G, d = s["q"].double(), case["block"], case["Hkv"], case["G"], case["d"]
        out = torch.zeros_like(q)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
        for i, n in enumerate(s["lens"].tolist()):
            if n == 0:
                continue
            ids = s["table"][i, :_up(n, ps)].long()
            K, V = ((c.view(torch.uint8)[ids].view(E4M3).double().unflatten(2, (-1, B)) * f[ids].double()[..., None, None])
                    .flatten(2, 3).permute(1, 0, 2, 3).reshape(H, -1, d)[:, :n] for c, f in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
            sc = torch.einsum("hgd,hnd->hgn", q[i].reshape(H, G, d), K) * s["scale"]
            z = torch.logsumexp(sc, -1)
            out[i] = torch.einsum("hgn,hnd->hgd", torch.exp(sc - z[..., None]), V).reshape(H * G, d)
            lse[i] = z.reshape(-1)
        return out, lse
    if op == "resize":
        return None
    pools = [p.double() for p in s["pools"]]
    if op == "fork":
        free = [i for i, r in enumerate(s["refs"].tolist()) if r == 0]
        moves = [(int(s["table"][a, n // ps]), None) for a in s["src"].tolist() for n in (int(s["lens"][a]),) if n % ps]
        moves = [(a, free[i]) for i, (a, _) in enumerate(moves)]
    else:
        refs = s["refs"].tolist()
        live = sum(r != 0 for r in refs)
        moves = list(zip([i for i in range(live, len(refs)) if refs[i]], [i for i in range(live) if not refs[i]]))
    for a, b in moves:
        for p in pools:
            p[b] = p[a]
    return [pools] + [None] * 4
