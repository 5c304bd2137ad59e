"""The layer operators under CUDA graph capture (their launches are programmatic
dependents of one another): one decode step of each, and the prefill with its
segments, captured once and replayed on new inputs; every replay must equal the
eager calls bit for bit."""
import pytest
import torch

from gated_delta_rule_46_gb300 import decay_decode, decay_prefill, linear, paged_append, paged_decode
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=g.device)


def test_decode_step_in_a_graph():
    """linear -> paged_append -> paged_decode -> linear -> decay_decode -> linear."""
    dev = need_gpu()
    N, H, D, ps = 5, 4, 128, 16
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    w = [(_randn(g, n, H * D) / 22).to(BF) for n in (3 * H * D, H * D, 3 * H * D, H * D)]
    ld = -torch.rand(H, generator=g, device=dev)
    table = torch.randperm(N * 20, generator=g, device=dev).to(torch.int32).reshape(N, 20)
    x = torch.empty(N, H * D, dtype=BF, device=dev)
    start = torch.tensor([0, 17, 200, 300, 64], dtype=torch.int32, device=dev)
    lens = start + 1
    state = {"kc": _randn(g, N * 20, H, ps, D).to(BF), "vc": _randn(g, N * 20, H, ps, D).to(BF),
             "pool": 0.1 * _randn(g, N, H, D, D)}

    def body():
        q, k, v = (t.unflatten(1, (H, D)) for t in linear(x, w[0]).split(H * D, 1))
        paged_append(k, v, state["kc"], state["vc"], table, start)
        y = linear(paged_decode(q, state["kc"], state["vc"], table, lens).reshape(N, -1), w[1], residual=x)
        q, k, v = (t.unflatten(1, (H, D)) for t in linear(y, w[2], act="silu").split(H * D, 1))
        return linear(decay_decode(q, k, v, ld, state["pool"]).reshape(N, -1), w[3], residual=y)

    x.copy_(_randn(g, N, H * D))
    body()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = body()
    for _ in range(3):
        x.copy_(_randn(g, N, H * D))
        before = {n: t.clone() for n, t in state.items()}
        graph.replay()
        torch.cuda.synchronize()
        got, after = out.clone(), {n: t.clone() for n, t in state.items()}
        for n, t in state.items():
            t.copy_(before[n])
        assert torch.equal(body(), got)
        assert all(torch.equal(state[n], after[n]) for n in state)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (torch.float32, 64)])
@pytest.mark.parametrize("lens,H", [([1500], 2), ([100] * 90, 4)])
def test_prefill_in_a_graph(dtype, d, lens, H):
    """Few chains (segments, three launches) and many (a schedule, then one kernel)."""
    dev = need_gpu()
    g = torch.Generator(device=dev)
    g.manual_seed(2)
    T = sum(lens)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    q, k, v = (torch.empty(T, H, d, dtype=dtype, device=dev) for _ in range(3))
    ld = -torch.rand(H, generator=g, device=dev) / 8
    s0 = torch.empty(len(lens), H, d, d, device=dev)

    def new():
        for t in (q, k, v, s0):
            t.copy_(0.3 * _randn(g, *t.shape))

    new()
    decay_prefill(q, k, v, ld, cu, s0)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, fin = decay_prefill(q, k, v, ld, cu, s0)
    for _ in range(3):
        new()
        graph.replay()
        torch.cuda.synchronize()
        o, f = decay_prefill(q, k, v, ld, cu, s0)
        assert torch.equal(o, out) and torch.equal(f, fin)
