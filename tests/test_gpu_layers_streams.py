"""Calls on another stream than torch's current one, beside work that is still queued
there: what they allocate must not be memory that the current stream has freed but
not finished with, nor go back to their own stream while the current one reads it."""
import pytest
import torch

from gated_delta_rule_46_gb300 import decay_decode, decay_prefill, linear, paged_decode
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DELAY = 200_000_000          # cycles, about a tenth of a second


def _calls(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    x, w = rnd(2048, 256).to(BF), rnd(1024, 256).to(BF)
    q, k, v = (0.3 * rnd(4096, 4, 128).to(BF) for _ in range(3))
    ld, cu = -torch.rand(4, generator=g, device=dev), torch.tensor([0, 4096], dtype=torch.int32, device=dev)
    pool = rnd(4096, 4, 32, 32)
    q1 = 0.3 * rnd(4096, 4, 32)
    kc, vc = rnd(512, 8, 64, 128).to(BF), rnd(512, 8, 64, 128).to(BF)
    table = torch.randperm(512, generator=torch.Generator().manual_seed(2)).to(torch.int32).reshape(4, 128).to(dev)
    lens = torch.tensor([8000, 5, 8192, 700], dtype=torch.int32, device=dev)
    qa = rnd(4, 256, 128).to(BF)
    return {
        "linear": lambda **kw: [linear(x, w, **kw)],
        "decay_prefill": lambda **kw: list(decay_prefill(q, k, v, ld, cu, **kw)),
        "decay_decode": lambda **kw: [decay_decode(q1, q1, q1, ld, pool.clone() if not kw else pool, **kw)],
        "paged_decode": lambda **kw: list(paged_decode(qa, kc, vc, table, lens, return_lse=True, **kw)),
    }


@pytest.mark.parametrize("name", ["linear", "decay_prefill", "decay_decode", "paged_decode"])
def test_memory_that_the_current_stream_still_uses(name):
    dev = need_gpu()
    call = _calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # freed here in blocks large and small, all still to be read after the delay
    freed = [torch.full((n,), 3, dtype=torch.int32, device=dev) for n in [1 << 24] + [1 << 20] * 4 + [1 << 14] * 64 + [128] * 64]
    kept = [torch.empty_like(t) for t in freed]
    torch.cuda.synchronize()
    torch.cuda._sleep(DELAY)
    for a, b in zip(kept, freed):
        a.copy_(b)
    del freed, b
    got = call(stream=s)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept), "the call wrote what the current stream was still to read"
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", ["linear", "decay_prefill", "decay_decode", "paged_decode"])
def test_results_that_the_current_stream_still_reads(name):
    dev = need_gpu()
    call = _calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(stream=s)
    sizes = [t.numel() * t.element_size() for t in got]
    kept = [torch.empty_like(t) for t in got]
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(DELAY)
    for a, b in zip(kept, got):
        a.copy_(b)
    del got, b
    with torch.cuda.stream(s):
        other = [torch.full((n,), 7, dtype=torch.uint8, device=dev) for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want)) and len(other)


def _args(name, dev):
    """The call with copies of its inputs, and these copies."""
    g = torch.Generator(device=dev).manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device=dev)  # noqa: E731
    if name == "linear":
        return linear, [rnd(2048, 256).to(BF), rnd(1024, 256).to(BF), rnd(1024), rnd(2048, 1024).to(BF)]
    if name == "decay_prefill":
        return (lambda *a, **kw: decay_prefill(*a, want_final_state=False, **kw)[0],
                [0.3 * rnd(4096, 4, 128).to(BF) for _ in range(3)] +
                [-rnd(4).abs(), torch.tensor([0, 4096], dtype=torch.int32, device=dev), rnd(1, 4, 128, 128)])
    if name == "decay_decode":
        return decay_decode, [0.3 * rnd(2048, 4, 64) for _ in range(3)] + [-rnd(4).abs(), rnd(2048, 4, 64, 64),
                                                                           torch.arange(2048, dtype=torch.int32, device=dev)]
    table = torch.randperm(512, generator=torch.Generator().manual_seed(2)).to(torch.int32).reshape(4, 128).to(dev)
    return paged_decode, [rnd(4, 256, 128).to(BF), rnd(512, 8, 64, 128).to(BF), rnd(512, 8, 64, 128).to(BF), table,
                          torch.tensor([8000, 5, 8192, 700], dtype=torch.int32, device=dev)]


@pytest.mark.parametrize("name", ["linear", "decay_prefill", "decay_decode", "paged_decode"])
def test_inputs_that_are_dropped_before_the_call_has_run(name):
    dev = need_gpu()
    f, args = _args(name, dev)
    want = f(*(t.clone() for t in args)).clone()
    s = torch.cuda.Stream()
    given = [t.clone() for t in args]
    sizes = [t.numel() * t.element_size() for t in given]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(DELAY)
    got = f(*given, stream=s)
    del given
    other = [torch.full((n,), 255, dtype=torch.uint8, device=dev) for n in sizes for _ in range(2)]     # NaN as numbers
    torch.cuda.synchronize()
    assert torch.equal(got, want) and len(other)
