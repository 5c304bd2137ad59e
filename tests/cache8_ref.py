"""Plain 64-bit forms of the cache in 8 bits and of its pages, from their definitions, on the CPU.

Codes and scales are exact: scales are powers of two, so a code is its value rounded
once, and nothing is left to a tolerance.  Attention over such a cache (``decode``)
rounds a float32 result as ``layers_ref`` says; a bf16 result is rounded once, by
at most 2^-8 of itself, and each softmax weight, which takes the tensor cores'
8-bit products in two parts of four significant bits, by at most 2^-8 of itself:
2^-7 in all.
"""
import math

import torch

import layers_ref

E4M3 = torch.float8_e4m3fn
F32_TOL = layers_ref.F32_TOL
BF16_TOL = 2.0 ** -7


def round_e4m3(y):
    """Four significant bits, no exponent below -6, ties to the even value; not finite: NaN."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.where(y.abs() < math.inf, torch.round(y / step) * step, math.nan)


def scale_for(amax):
    s = 2.0 ** -126
    while 448 * s < amax:
        s *= 2
    return s


def append(x, code, scale, table, start, lens):
    """x [T, H, d] into code [P, H, ps, d] and scale [P, H, ps / B], both float64, in place."""
    P, H, ps, d = code.shape
    B = ps // scale.shape[2]
    t = 0
    for i, n in enumerate(lens):
        done = 0
        while done < n:
            pos = start[i] + done
            m, r, page = min(B - pos % B, n - done), pos % B, int(table[i][pos // ps])
            b = pos % ps // B
            for h in range(H):
                y = x[t + done:t + done + m, h].double()
                fine = y[torch.isfinite(y)]
                s = scale_for(float(fine.abs().max()) if fine.numel() else 0.0)
                rows = code[page, h, b * B:(b + 1) * B]
                if r:
                    was = float(scale[page, h, b])
                    s = max(s, 2.0 ** math.ceil(math.log2(was)))
                    if s != was:
                        rows[:r] = round_e4m3(rows[:r] * was / s)
                scale[page, h, b] = s
                rows[r:r + m] = round_e4m3(y / s)
            done += m
        t += n


def values(code, scale):
    """The values that codes [P, H, ps, d] and scales [P, H, ps / B] stand for, in float64."""
    B = code.shape[2] // scale.shape[2]
    return code.double() * scale.double().repeat_interleave(B, 2)[..., None]


def decode(q, code_k, code_v, scale_k, scale_v, table, lens, scale):
    return layers_ref.paged(q, values(code_k, scale_k), values(code_v, scale_v), table, lens, scale)


def close(name, got, ref):
    e, t = layers_ref.rel(got, ref), BF16_TOL if got.dtype == torch.bfloat16 else F32_TOL
    assert e <= t, f"{name}: rel-L2 {e:.3e} > {t:.3e}"


def same(name, got, ref):
    """Codes or scales: the same values, NaN in the same places."""
    g, r = got.detach().cpu().double(), ref.double()
    assert torch.equal(torch.isnan(g), torch.isnan(r)), f"{name}: NaN in other places"
    bad = (g != r) & ~torch.isnan(r)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}: " \
                          f"{g[bad][0].item()} for {r[bad][0].item()}"


class Pages:
    """Page table, pages held and holders, as the calls define them."""

    def __init__(self, rows, cols, pages, ps):
        self.table = [[-1] * cols for _ in range(rows)]
        self.held, self.refs, self.ps, self.cols = [0] * rows, [0] * pages, ps, cols
        self.errors = set()

    def free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def resize(self, tokens):
        want = {}
        for i, t in enumerate(tokens):
            w = self.held[i] if t < 0 else -(-t // self.ps)
            if w > self.cols or not 0 <= self.held[i] <= self.cols:
                self.errors.add("arg")
                w = None
            want[i] = w
        for i, w in want.items():
            if w is not None and w < self.held[i]:
                for e in range(w, self.held[i]):
                    p, self.table[i][e] = self.table[i][e], -1
                    if p >= len(self.refs) or (p >= 0 and self.refs[p] == 0):
                        self.errors.add("arg")
                    elif p >= 0 and self.refs[p] > 0:
                        self.refs[p] -= 1
                self.held[i] = w
        free = self.free()
        for i, w in want.items():
            while w is not None and self.held[i] < w:
                if not free:
                    self.errors.add("pages")
                    break
                p = free.pop(0)
                self.table[i][self.held[i]], self.refs[p] = p, 1
                self.held[i] += 1

    def fork(self, pools, lens, src, dst):
        """pools: lists of tensors [P, ...], changed in place."""
        N, free, copies, taken = len(self.table), self.free(), [], []
        pairs = [(a, b) for a, b in zip(src, dst)]
        inside = lambda a, b: 0 <= a < N and 0 <= b < N  # noqa: E731
        sources = {a for a, b in pairs if inside(a, b)}
        rows = []
        seen = set()
        for a, b in pairs:
            if a < 0 or b < 0:
                continue
            if not inside(a, b):
                self.errors.add("arg")
                continue
            ok = b not in sources and b not in seen and self.held[b] == 0
            seen.add(b)
            n = lens[a]
            ok = ok and 0 <= self.held[a] <= self.cols and 0 <= n <= self.held[a] * self.ps
            if ok and n % self.ps:
                p = self.table[a][n // self.ps]
                ok = 0 <= p < len(self.refs) and self.refs[p] != 0
            if not ok:
                self.errors.add("arg")
                continue
            new = None
            if n % self.ps:
                if not free:
                    self.errors.add("pages")
                    continue
                new = free.pop(0)
                copies.append((self.table[a][n // self.ps], new))
            rows.append((a, b, n, new))
        for a, b, n, new in rows:
            for e in range(n // self.ps):
                p = self.table[a][e]
                if 0 <= p < len(self.refs):
                    self.refs[p] += self.refs[p] >= 0
                else:
                    self.errors.add("arg")
                    p = -1
                self.table[b][e] = p
            if new is not None:
                self.table[b][n // self.ps] = new
                taken.append(new)
            self.held[b], lens[b] = -(-n // self.ps), n
        for p in taken:
            self.refs[p] = 1
        for x in pools:
            for a, b in copies:
                x[b] = x[a]

    def compact(self, pools):
        """Returns the new ids of all pages."""
        live = sum(r != 0 for r in self.refs)
        holes = [p for p in range(live) if self.refs[p] == 0]
        movers = [p for p in range(live, len(self.refs)) if self.refs[p] != 0]
        to = [p if r else -1 for p, r in enumerate(self.refs)]
        for a, b in zip(movers, holes):
            to[a], self.refs[b], self.refs[a] = b, self.refs[a], 0
            for x in pools:
                x[b] = x[a]
        for row in self.table:
            for e, p in enumerate(row):
                if p >= 0:
                    row[e] = to[p] if p < len(to) else -1
                    if row[e] < 0:
                        self.errors.add("arg")
        return to, live
