"""An expired bounded wait in the layer operators' tensor-core kernels: the call
returns, KDA_ERR_DEVICE_TIMEOUT is in the status word, the context stays usable
and the next call is exact.  kda_testing_expire_next_wait makes one role of CTA 0
give up; nothing faults, traps or hangs."""
import pytest
import torch

import layers_ref as ref
from gated_delta_rule_46_gb300 import check_device_status, decay_prefill, kda, linear, paged_decode
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
expire_next_wait = kda.testing_expire_next_wait


def _twice(bit, call, check):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    expire_next_wait(bit)
    call(status)
    assert check_device_status(status) == kda.KDA_ERR_DEVICE_TIMEOUT
    torch.cuda.synchronize()                       # raises if the context had an error
    status.zero_()
    got = call(status)
    assert check_device_status(status) == kda.KDA_OK
    check(got)


@pytest.mark.parametrize("M,N,K,ld", [(40, 1024, 2048, 2048), (300, 264, 256, 257), (700, 4096, 256, 256), (700, 2048, 256, 256)])
def test_linear(M, N, K, ld):
    """Split K over clusters; element-wise loads; both pair tiles."""
    dev = need_gpu()
    g = torch.Generator().manual_seed(1)
    x, w = torch.randn(M, ld, generator=g).to(BF)[:, :K], (torch.randn(N, K, generator=g) / K ** 0.5).to(BF)
    xd, wd = torch.empty(M, ld, dtype=BF, device=dev)[:, :K].copy_(x), w.to(dev)
    _twice(kda.KDA_TESTING_LINEAR, lambda s: linear(xd, wd, status=s),
           lambda y: ref.close("out", y, ref.linear(x, w, None, None, "none")))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,H", [([3000, 900], 2), ([70] * 100, 2)])
def test_decay_prefill(d, lens, H):
    """With segments and without."""
    dev = need_gpu()
    g = torch.Generator().manual_seed(2)
    T = sum(lens)
    q, k, v = ((torch.randn(T, H, d, generator=g) / d ** 0.25).to(BF) for _ in range(3))
    ld = -torch.rand(H, generator=g)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=dev)
    args = [t.to(dev) for t in (q, k, v, ld)]

    def check(got):
        ro, rf = ref.decay(q, k, v, ld, lens)
        ref.close("out", got[0], ro)
        ref.close("state", got[1], rf)
    _twice(kda.KDA_TESTING_DECAY, lambda s: decay_prefill(*args, cu, status=s), check)


@pytest.mark.parametrize("d", [64, 128])
def test_paged_decode(d):
    dev = need_gpu()
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.randn(40, 2, 32, d, generator=g).to(BF) for _ in range(2))
    q = torch.randn(2, 8, d, generator=g).to(BF)
    table, lens = torch.randperm(40, generator=g).to(torch.int32).reshape(2, 20), [620, 33]
    args = [t.to(dev) for t in (q, kc, vc, table, torch.tensor(lens, dtype=torch.int32))]

    def check(got):
        ref.close("out", got, ref.paged(q, kc, vc, table, lens, d ** -0.5)[0])
    _twice(kda.KDA_TESTING_PAGED, lambda s: paged_decode(*args, status=s), check)


def test_bits_are_taken_by_their_own_operator():
    """An armed bit of one operator leaves the others' calls alone, and 0 disarms."""
    dev = need_gpu()
    x, w = torch.randn(8, 64, device=dev).to(BF), torch.randn(64, 64, device=dev).to(BF)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    expire_next_wait(kda.KDA_TESTING_PAGED | kda.KDA_TESTING_DECAY)
    a = linear(x, w, status=status)
    expire_next_wait(0)
    b = linear(x, w, status=status)
    assert check_device_status(status) == kda.KDA_OK and torch.equal(a, b)
