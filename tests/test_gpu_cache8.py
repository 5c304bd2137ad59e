"""A cache in 8 bits as it is served: pages handed out, prompts and single tokens appended, attention over them, rows
forked, cut back and ended, pages moved together; captured in graphs, on other streams, beside queued work."""
import math
import random

import pytest
import torch

import cache8_ref as ref
from gated_delta_rule_46_gb300 import (check_device_status, kda, paged_append_q8, paged_decode_q8, pages_compact, pages_fork,
                                       pages_resize)
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF, F32, E4M3 = torch.bfloat16, torch.float32, ref.E4M3
DELAY = 200_000_000          # cycles, about a tenth of a second


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Served:
    """A batch on the device, and beside it each row's own cache of one long page in float64."""

    def __init__(self, rows, cols, pages, ps, B, H, G, d, dtype, dev, seed):
        self.dev, self.ps, self.B, self.H, self.G, self.d, self.dtype = dev, ps, B, H, G, d, dtype
        self.g = torch.Generator().manual_seed(seed)
        u8 = torch.full((pages, H, ps, d), 0x7F, dtype=torch.uint8, device=dev)          # nobody clears a page: NaN
        self.kc, self.vc = u8.view(E4M3), u8.clone().view(E4M3)
        self.ks, self.vs = (torch.full((pages, H, ps // B), math.nan, device=dev) for _ in range(2))
        self.table = torch.full((rows, cols), -1, dtype=torch.int32, device=dev)
        self.held, self.refs = _i32([0] * rows, dev), _i32([0] * pages, dev)
        self.lens, self.dlens = [0] * rows, _i32([0] * rows, dev)
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        self.own = [[torch.zeros(1, H, cols * ps, d, dtype=torch.float64), torch.ones(1, H, cols * ps // B, dtype=torch.float64),
                     torch.zeros(1, H, cols * ps, d, dtype=torch.float64), torch.ones(1, H, cols * ps // B, dtype=torch.float64)]
                    for _ in range(rows)]

    def pools(self):
        return [self.kc, self.vc, self.ks, self.vs]

    def ok(self):
        assert check_device_status(self.status) == kda.KDA_OK
        assert self.held.tolist() == [-(-n // self.ps) for n in self.lens]

    def resize(self, lens):
        pages_resize(self.table, self.held, self.refs, _i32(lens, self.dev), self.ps, status=self.status)
        self.lens = list(lens)
        self.dlens.copy_(_i32(lens, self.dev))
        self.ok()

    def append(self, new):
        """new[i] tokens more for row i."""
        start = list(self.lens)
        self.resize([a + b for a, b in zip(start, new)])
        T = sum(new)
        k, v = ((torch.randn(T, self.H, self.d, generator=self.g) * torch.exp(torch.randn(T, self.H, 1, generator=self.g)))
                .to(self.dtype) for _ in range(2))
        one = all(n == 1 for n in new)
        cu = None if one else _i32([0] + torch.tensor(new).cumsum(0).tolist(), self.dev)
        paged_append_q8(k.to(self.dev), v.to(self.dev), self.kc, self.vc, self.ks, self.vs, self.table, _i32(start, self.dev),
                        cu_seqlens=cu, status=self.status)
        t = 0
        for i, n in enumerate(new):
            kc, ks, vc, vs = self.own[i]
            ref.append(k[t:t + n], kc, ks, [[0]], [start[i]], [n])
            ref.append(v[t:t + n], vc, vs, [[0]], [start[i]], [n])
            t += n

    def attend(self):
        q = torch.randn(len(self.lens), self.H * self.G, self.d, generator=self.g).to(self.dtype)
        out, lse = paged_decode_q8(q.to(self.dev), self.kc, self.vc, self.ks, self.vs, self.table, self.dlens, return_lse=True,
                                   status=self.status)
        self.ok()
        for i, n in enumerate(self.lens):
            kc, ks, vc, vs = self.own[i]
            want, z = ref.decode(q[i:i + 1], kc, vc, ks, vs, torch.zeros(1, 1, dtype=torch.int32), [n], self.d ** -0.5)
            if n == 0:
                assert not out[i].any() and torch.isneginf(lse[i]).all()
                continue
            ref.close(f"row {i} of {n} tokens", out[i:i + 1], want)
            # scores are sums of d products with at most 2^-18 of the largest factors' product missing, or float32's own error
            assert float((lse[i].double().cpu() - z[0]).abs().max()) < 1e-3

    def fork(self, src, dst):
        pages_fork(self.pools(), self.table, self.held, self.refs, self.dlens, _i32(src, self.dev), _i32(dst, self.dev), self.ps,
                   status=self.status)
        for a, b in zip(src, dst):
            self.lens[b] = self.lens[a]
            self.own[b] = [t.clone() for t in self.own[a]]
        self.ok()
        assert self.dlens.tolist() == self.lens

    def compact(self):
        to, live = pages_compact(self.pools(), self.table, self.refs, status=self.status)
        n = int(live)
        self.ok()
        assert n == len({p for p in self.table.flatten().tolist() if p >= 0}) and bool((self.refs[:n] > 0).all())
        assert not self.refs[n:].any() and int(self.table.max()) == n - 1


@pytest.mark.parametrize("dtype,d,G,ps,B", [(BF, 128, 4, 64, 16), (BF, 64, 16, 32, 32), (BF, 32, 3, 16, 16), (BF, 64, 20, 64, 64),
                                            (F32, 64, 2, 32, 16), (F32, 128, 9, 64, 64)])
def test_a_served_batch(dtype, d, G, ps, B):
    dev = need_gpu()
    rows, r = 7, random.Random(d + G)
    s = Served(rows, 12, 40, ps, B, 2, G, d, dtype, dev, d + G)
    s.append([ps * 3 + 5, 1, ps, 0, 2 * ps - 1, 0, 0])                   # prompts
    s.attend()
    s.fork([0, 0, 4], [3, 5, 6])                                         # samples that go on from two of them
    s.attend()
    for _ in range(3):
        s.append([1] * rows)
        s.attend()
    s.resize([0, s.lens[1], 0, s.lens[3], s.lens[4], s.lens[5], 0])      # some end
    s.compact()
    s.attend()
    s.append([r.randrange(2 * ps) for _ in range(rows)])                 # prompts in their place, and chunks of the others'
    s.attend()
    # drafts cut back: to a whole page, or into a page of the row's own
    s.resize([max(0, n - 3) if int(s.refs[s.table[i, (n - 4) // ps].long()]) == 1 else n // ps * ps if n > 3 else 0
              for i, n in enumerate(s.lens)])
    s.append([1] * rows)
    s.compact()
    s.attend()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_decoding_loop_in_a_graph(dtype):
    """Rows that grow, take pages and attend, captured once: every replay as the eager calls, bit for bit."""
    dev = need_gpu()
    N, H, G, d, ps, cols = 5, 2, 4, 64, 16, 12
    P = N * cols
    g = torch.Generator(device=dev).manual_seed(1)
    lens = _i32([15, 0, 16, 31, 100], dev)
    table = torch.full((N, cols), -1, dtype=torch.int32, device=dev)
    held, refs = _i32([0] * N, dev), _i32([0] * P, dev)
    pages_resize(table, held, refs, lens, ps)
    kc, vc = (torch.zeros(P, H, ps, d, dtype=torch.uint8, device=dev).view(E4M3) for _ in range(2))
    ks, vs = torch.ones(P, H, 1, device=dev), torch.ones(P, H, 1, device=dev)
    x = torch.empty(N, (G + 2) * H * d, dtype=dtype, device=dev)
    state = [lens, table, held, refs, kc.view(torch.uint8), vc.view(torch.uint8), ks, vs]

    def body():
        q, k, v = x[:, :G * H * d].unflatten(1, (G * H, d)), *(t.unflatten(1, (H, d)) for t in x[:, G * H * d:].split(H * d, 1))
        start = lens.clone()
        lens.add_(1)
        pages_resize(table, held, refs, lens, ps)
        paged_append_q8(k, v, kc, vc, ks, vs, table, start)
        return paged_decode_q8(q, kc, vc, ks, vs, table, lens, return_lse=True)

    def new():
        x.copy_(torch.randn(x.shape, generator=g, device=dev))

    new()
    first = [t.clone() for t in state]
    body()
    torch.cuda.synchronize()
    for t, f in zip(state, first):
        t.copy_(f)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = body()
    for _ in range(40):
        new()
        before = [t.clone() for t in state]
        graph.replay()
        torch.cuda.synchronize()
        got, after = [t.clone() for t in out], [t.clone() for t in state]
        for t, b in zip(state, before):
            t.copy_(b)
        want = body()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(after, state))
    assert held.tolist() == [-(-n // ps) for n in lens.tolist()]


def _cache(dev, g, P=512, H=8, ps=64, d=128, B=16):
    code = lambda: (torch.randn(P, H, ps, d, generator=g, device=dev) * 60).clamp(-440, 440).to(E4M3)  # noqa: E731
    scale = lambda: torch.exp2(torch.randint(-8, -2, (P, H, ps // B), generator=g, device=dev).float())  # noqa: E731
    return code(), code(), scale(), scale()


def _calls(name, dev):
    """The call with its arguments (which it may update), and the outputs to compare."""
    g = torch.Generator(device=dev).manual_seed(3)
    table = torch.randperm(512, generator=torch.Generator().manual_seed(2)).to(torch.int32).reshape(4, 128).to(dev)
    if name == "append":
        k, v = (torch.randn(4000, 8, 128, generator=g, device=dev).to(BF) for _ in range(2))
        args = [k, v, *_cache(dev, g), table, _i32([5, 100, 0, 700], dev), _i32([0, 1000, 1001, 3500, 4000], dev)]
        return lambda a, **kw: paged_append_q8(*a, **kw) or a[2:6], args
    if name == "decode":
        args = [torch.randn(4, 32, 128, generator=g, device=dev).to(BF), *_cache(dev, g), table, _i32([8000, 5, 8192, 700], dev)]
        return lambda a, **kw: list(paged_decode_q8(*a, return_lse=True, **kw)), args
    if name == "resize":
        refs = torch.zeros(70000, dtype=torch.int32, device=dev)
        refs[:512] = 1
        t = torch.full((4, 20000), -1, dtype=torch.int32, device=dev)
        t[:, :128] = table
        args = [t, _i32([128] * 4, dev), refs, _i32([16 * 17000, 0, 16 * 100, 16 * 15000], dev)]
        return lambda a, **kw: pages_resize(*a, 16, **kw) or a[:3], args
    pools = list(_cache(dev, g))
    refs = torch.zeros(512, dtype=torch.int32, device=dev)
    t = torch.full((8, 64), -1, dtype=torch.int32, device=dev)
    if name == "fork":
        t[:4, :50] = table[:, :50]
        refs[table[:, :50].flatten().long()] = 1
        lens = _i32([50 * 64 - 5, 64 * 49 + 1, 50 * 64, 50 * 64 - 60, 0, 0, 0, 0], dev)
        args = [*pools, t, _i32([50] * 4 + [0] * 4, dev), refs, lens, _i32([0, 1, 2, 0], dev), _i32([7, 5, 4, 6], dev)]
        return lambda a, **kw: pages_fork(a[:4], *a[4:], 64, **kw) or a[:8], args
    t[:4] = table[:, 64:]
    refs[table[:, 64:].flatten().long()] = 1
    return lambda a, **kw: [*pages_compact(a[:4], a[4], a[5], **kw), *a], [*pools, t, refs]


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


NAMES = ["append", "decode", "resize", "fork", "compact"]


@pytest.mark.parametrize("name", NAMES)
def test_inputs_that_are_dropped_before_the_call_has_run(name):
    dev = need_gpu()
    f, args = _calls(name, dev)
    want = [_bytes(t).clone() for t in f([t.clone() for t in args])]
    s = torch.cuda.Stream()
    given = [t.clone() for t in args]
    sizes = [t.numel() * t.element_size() for t in given]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    got = f(given, stream=s)
    updated = {t.data_ptr() for t in got}
    dropped = [n for t, n in zip(given, sizes) if t.data_ptr() not in updated]
    del given
    other = [torch.full((n,), 255, dtype=torch.uint8, device=dev) for n in dropped for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(_bytes(a), b) for a, b in zip(got, want)) and len(other) == 2 * len(dropped)


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name):
    dev = need_gpu()
    f, args = _calls(name, dev)
    want = [_bytes(t).clone() for t in f([t.clone() for t in args])]
    given = [t.clone() for t in args]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.full((n,), 3, dtype=torch.int32, device=dev) for n in [1 << 20] * 4 + [1 << 14] * 64 + [128] * 64]
    kept = [torch.empty_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    for a, b in zip(kept, freed):
        a.copy_(b)
    del freed, b
    got = f(given, stream=s)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept), "the call wrote what the current stream was still to read"
    assert all(torch.equal(_bytes(a), b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_captured_calls_replayed_at_once(name):
    """Two captured calls on states of their own, replayed on two streams at a time, as one after the other."""
    dev = need_gpu()
    f, args = _calls(name, dev)
    states = [[t.clone() for t in args] for _ in range(2)]
    f([t.clone() for t in args])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for a in states:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f(a))
        graphs.append(g)
    want = [_bytes(t).clone() for t in f([t.clone() for t in args])]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for a in states:
            for t, x in zip(a, args):
                _bytes(t).copy_(_bytes(x))
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(_bytes(a), b) for a, b in zip(out, want))


@pytest.mark.parametrize("d,G", [(128, 4), (64, 16), (32, 20)])
def test_a_wait_that_expires(d, G):
    """The call returns, the status word says so, and the next call is right."""
    dev = need_gpu()
    g = torch.Generator().manual_seed(3)
    P, H, ps, B = 40, 2, 32, 16
    kc, vc = (torch.randn(P, H, ps, d, generator=g).to(E4M3) for _ in range(2))
    ks, vs = (torch.exp2(torch.randint(-2, 2, (P, H, ps // B), generator=g).float()) for _ in range(2))
    q = torch.randn(2, H * G, d, generator=g).to(BF)
    table, lens = torch.randperm(P, generator=g).to(torch.int32).reshape(2, 20), [620, 33]
    args = [t.to(dev) for t in (q, kc, vc, ks, vs, table, torch.tensor(lens, dtype=torch.int32))]
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kda.testing_expire_next_wait(kda.KDA_TESTING_PAGED)
    paged_decode_q8(*args, status=status)
    assert check_device_status(status) == kda.KDA_ERR_DEVICE_TIMEOUT
    torch.cuda.synchronize()
    status.zero_()
    got = paged_decode_q8(*args, status=status)
    assert check_device_status(status) == kda.KDA_OK
    ref.close("out", got, ref.decode(q, kc, vc, ks, vs, table, lens, d ** -0.5)[0])


def test_rows_and_pages_past_32_bits():
    """A cache whose byte offsets pass 2^32, read and written at its end."""
    dev = need_gpu()
    P, H, ps, d, B = 40000, 8, 128, 128, 64                              # 5.2 GB of keys, as much of values
    code = torch.zeros(2, P, H, ps, d, dtype=torch.uint8, device=dev)
    kc, vc = code[0].view(E4M3), code[1].view(E4M3)
    ks, vs = torch.ones(P, H, ps // B, device=dev), torch.ones(P, H, ps // B, device=dev)
    g = torch.Generator().manual_seed(6)
    k, v = (torch.randn(200, H, d, generator=g).to(BF) for _ in range(2))
    table = _i32([[P - 1, P - 2]], dev)
    paged_append_q8(k.to(dev), v.to(dev), kc, vc, ks, vs, table, _i32([0], dev), cu_seqlens=_i32([0, 200], dev))
    own = [torch.zeros(2, H, ps, d, dtype=torch.float64), torch.ones(2, H, ps // B, dtype=torch.float64),
           torch.zeros(2, H, ps, d, dtype=torch.float64), torch.ones(2, H, ps // B, dtype=torch.float64)]
    ref.append(k, own[0], own[1], [[1, 0]], [0], [200])
    ref.append(v, own[2], own[3], [[1, 0]], [0], [200])
    ref.same("keys", kc[P - 2:], own[0])
    ref.same("values", vc[P - 2:], own[2])
    for dtype in (BF, F32):
        q = torch.randn(1, 2 * H, d, generator=g).to(dtype)
        got = paged_decode_q8(q.to(dev), kc, vc, ks, vs, table, _i32([200], dev))
        ref.close("out", got, ref.decode(q, own[0], own[2], own[1], own[3], torch.tensor([[1, 0]]), [200], d ** -0.5)[0])
    refs = torch.zeros(P, dtype=torch.int32, device=dev)
    refs[P - 2:] = 1
    pages_compact([kc, vc, ks, vs], table, refs)
    assert table.tolist() == [[1, 0]]
    ref.same("keys", kc[:2], own[0])
    ref.same("values", vc[:2], own[2])
