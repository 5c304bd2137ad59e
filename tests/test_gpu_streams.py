"""The KDA calls on another stream than torch's current one, beside work that is still
queued there (as tests/test_gpu_layers_streams.py for the operators around them)."""
import pytest
import torch

import gated_delta_rule_46_gb300 as K
from gated_delta_rule_46_gb300 import inputs
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
DELAY = 200_000_000          # cycles, about a tenth of a second


def _calls(dev):
    w = inputs.custom([3000, 1096], H=4, dk=128, dv=128, dtype=torch.bfloat16, init="randn0.1")
    d = {n: (t.to(dev) if t is not None else None) for n, t in inputs.prefill_inputs(w).items()}
    pre = [d[n] for n in ("q", "k", "v", "z", "A", "beta", "cu_seqlens")]
    g = K.gate(d["z"], d["A"])
    N = 512
    one = [d[n][:N].contiguous() for n in ("q", "k", "v", "z")]
    state = 0.1 * torch.randn(N, 4, 128, 128, generator=torch.Generator(device=dev).manual_seed(1), device=dev)
    M = 0.05 * torch.randn(3, 2, 4, 128, 128, generator=torch.Generator(device=dev).manual_seed(2), device=dev)
    return {
        "gate": lambda **kw: [K.gate(d["z"], d["A"], **kw)],
        "chunk_prefill": lambda **kw: list(K.chunk_prefill(*pre, d["initial_state"], **kw)),
        "chunk_prefill_logdecay": lambda **kw: list(
            K.chunk_prefill_logdecay(d["q"], d["k"], d["v"], g, d["beta"], d["cu_seqlens"], **kw)),
        "decode_step": lambda **kw: [K.decode_step(*one, d["A"], d["beta"][:N].contiguous(), state.clone() if not kw else state,
                                                   **kw)],
        "decode_tokens": lambda **kw: [K.decode_tokens(*(t.unsqueeze(1) for t in one), d["A"], d["beta"][:N].unsqueeze(1),
                                                       state.clone() if not kw else state, **kw)],
        "segment_map": lambda **kw: list(K.segment_map(*pre, **kw)),
        "state_compose": lambda **kw: [K.state_compose(M, M, **kw)],
    }


NAMES = ["gate", "chunk_prefill", "chunk_prefill_logdecay", "decode_step", "decode_tokens", "segment_map", "state_compose"]


@pytest.mark.parametrize("name", NAMES)
def test_memory_that_the_current_stream_still_uses(name):
    dev = need_gpu()
    call = _calls(dev)[name]
    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    # freed here in blocks large and small, all still to be read after the delay
    freed = [torch.full((n,), 3, dtype=torch.int32, device=dev) for n in [1 << 24] * 2 + [1 << 20] * 8 + [1 << 14] * 64]
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


@pytest.mark.parametrize("name", NAMES)
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


@pytest.mark.parametrize("name", ["chunk_prefill", "decode_tokens", "segment_map"])
def test_inputs_that_are_dropped_before_the_call_has_run(name):
    dev = need_gpu()
    w = inputs.custom([3000, 1096], H=4, dk=128, dv=128, dtype=torch.bfloat16)
    d = {n: (t.to(dev) if t is not None else None) for n, t in inputs.prefill_inputs(w).items()}
    order = [d[n] for n in ("q", "k", "v", "z", "A", "beta", "cu_seqlens")]
    f = {"chunk_prefill": lambda *a, **kw: K.chunk_prefill(*a, **kw)[0], "segment_map": lambda *a, **kw: K.segment_map(*a, **kw)[1],
         "decode_tokens": lambda *a, **kw: K.decode_tokens(*a, **kw)}[name]
    if name == "decode_tokens":
        order = [t[:1024].unsqueeze(1).contiguous() for t in order[:4]] + [d["A"], d["beta"][:1024].unsqueeze(1).contiguous(),
                                                                          torch.ones(1024, 4, 128, 128, device=dev)]
    want = f(*(t.clone() for t in order)).clone()
    s = torch.cuda.Stream()
    given = [t.clone() for t in order]
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
