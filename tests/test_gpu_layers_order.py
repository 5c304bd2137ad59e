"""Kernels of these operators may start before the one before them in the stream
has ended: back-to-back calls that write each other's inputs give, every time,
what the same calls give with a synchronisation between them."""
import torch

import pytest
from gated_delta_rule_46_gb300 import decay_decode, decay_prefill, linear, paged_append, paged_decode
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def _run(n, T, H, d, x, w, ld, cu, sync):
    """A segmented prefill between projections that overwrite its buffers, states handed on from call to call."""
    pause = torch.cuda.synchronize if sync else lambda: None
    qkv = torch.empty(T, 3 * H * d, dtype=BF, device=ld.device)
    out = torch.empty(T, H, d, dtype=BF, device=ld.device)
    state = torch.zeros(1, H, d, d, device=ld.device)
    kept = []
    for i in range(n):
        linear(x[i % 2], w[0], out=qkv)
        pause()
        q, k, v = (qkv[:, j * H * d:(j + 1) * H * d].unflatten(1, (H, d)) for j in range(3))
        decay_prefill(q, k, v, ld, cu, initial_state=state, final_state=state, out=out, scale=0.1)
        pause()
        y = linear(out.reshape(T, -1), w[1])
        pause()
        kept.append(y)
    return kept, state


@pytest.mark.parametrize("T,H,d", [(2048, 4, 128), (2048, 4, 64), (700, 2, 128), (4096, 16, 128)])
def test_prefill_between_projections(T, H, d):
    dev = need_gpu()
    g = torch.Generator().manual_seed(T + H)
    x = [torch.randn(T, 256, generator=g).to(BF).to(dev) for _ in range(2)]
    w = [(torch.randn(3 * H * d, 256, generator=g) / 64).to(BF).to(dev), (torch.randn(256, H * d, generator=g) / 64).to(BF).to(dev)]
    ld = (-torch.rand(H, generator=g) / 100).to(dev)
    cu = torch.tensor([0, T], dtype=torch.int32, device=dev)
    want, state = _run(12, T, H, d, x, w, ld, cu, True)
    for _ in range(5):
        got, last = _run(12, T, H, d, x, w, ld, cu, False)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(last, state)


def test_decode_steps_between_projections():
    """linear -> append -> attend -> linear -> decay step, the outputs of each the inputs of the next."""
    dev = need_gpu()
    N, H, d, ps = 8, 4, 64, 16
    g = torch.Generator().manual_seed(9)
    w = [(torch.randn(3 * H * d, H * d, generator=g) / 16).to(BF).to(dev) for _ in range(2)]
    x0 = torch.randn(N, H * d, generator=g).to(BF).to(dev)
    table = torch.arange(N * 8, dtype=torch.int32, device=dev).reshape(N, 8)
    ld = (-torch.rand(H, generator=g)).to(dev)

    def run(sync):
        pause = torch.cuda.synchronize if sync else lambda: None
        kc, vc = (torch.zeros(N * 8, H, ps, d, dtype=BF, device=dev) for _ in range(2))
        pool = torch.zeros(N, H, d, d, device=dev)
        lens = [torch.full((N,), i, dtype=torch.int32, device=dev) for i in range(101)]
        x = x0
        for i in range(100):
            qkv = linear(x, w[0], act="silu")
            pause()
            q, k, v = (qkv[:, j * H * d:(j + 1) * H * d].unflatten(1, (H, d)) for j in range(3))
            paged_append(k, v, kc, vc, table, lens[i])
            pause()
            y = paged_decode(q, kc, vc, table, lens[i + 1])
            pause()
            qkv = linear(y.reshape(N, -1), w[1], act="sigmoid")
            pause()
            q, k, v = (qkv[:, j * H * d:(j + 1) * H * d].unflatten(1, (H, d)) for j in range(3))
            x = decay_decode(q, k, v, ld, pool, scale=0.05).reshape(N, -1)
            pause()
        return x, pool, kc, vc
    want = run(True)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(run(False), want))
