"""decay_prefill in bf16 with head sizes that fill only a part of the tensor-core
tiles: neighbouring heads stay apart, segments, non-finite values, timeouts, and
the same sizes with rows that no 16-byte copy can start on."""
import pytest
import torch

import layers_ref as ref
from gated_delta_rule_46_gb300 import check_device_status, decay_prefill, kda
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
DIMS = [(32, 32), (32, 64), (64, 32), (32, 128), (128, 32), (64, 128), (128, 64)]


def _inputs(lens, H, dk, dv, seed):
    g = torch.Generator().manual_seed(seed)
    T = sum(lens)
    q, k = ((torch.randn(T, H, dk, generator=g) / dk ** 0.5).to(BF) for _ in range(2))
    v = torch.randn(T, H, dv, generator=g).to(BF)
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32)
    return q, k, v, -torch.exp2(-8 * torch.rand(H, generator=g)), cu, 0.1 * torch.randn(len(lens), H, dk, dv, generator=g)


@pytest.mark.parametrize("dk,dv", DIMS)
def test_heads_stay_apart(dk, dv):
    """NaN in one head's rows and state changes no bit of the heads beside it."""
    dev = need_gpu()
    args = [t.to(dev) for t in _inputs([200, 64, 7], 3, dk, dv, 1)]
    out, fin = decay_prefill(*args)
    for i in (0, 1, 2, 5):
        args[i][:, 1] = float("nan")
    out2, fin2 = decay_prefill(*args)
    for h in (0, 2):
        assert torch.equal(out2[:, h], out[:, h]) and torch.equal(fin2[:, h], fin[:, h])
    assert out2[:, 1].isnan().all() and fin2[:, 1].isnan().all()


@pytest.mark.parametrize("dk,dv", DIMS)
def test_a_later_infinity_stays_later(dk, dv):
    """An infinite value channel reaches its own token and later ones, in its channel alone."""
    dev = need_gpu()
    args = [t.to(dev) for t in _inputs([150], 2, dk, dv, 2)]
    out, _ = decay_prefill(*args)
    args[2][70, 1, dv - 3] = float("inf")
    out2, fin2 = decay_prefill(*args)
    clean = torch.ones(dv, dtype=torch.bool, device=dev)
    clean[dv - 3] = False
    assert torch.equal(out2[:, 0], out[:, 0]) and torch.equal(out2[:, 1][:, clean], out[:, 1][:, clean])
    ref.close("earlier tokens", out2[:70, 1, dv - 3], out[:70, 1, dv - 3].double().cpu())
    assert not out2[70:, 1, dv - 3].isfinite().any() and not fin2[0, 1, :, dv - 3].isfinite().any()


@pytest.mark.parametrize("dk,dv", DIMS)
@pytest.mark.parametrize("odd", [False, True])
def test_segments(dk, dv, odd):
    """Few long chains; with `odd` the rows start on odd elements, and run on the CUDA cores."""
    dev = need_gpu()
    lens = [2100, 0, 900]
    q, k, v, ld, cu, init = _inputs(lens, 2, dk, dv, 3)
    ld = ld / 256
    ro, rf = ref.decay(q, k, v, ld, lens, init)

    def place(t):
        T, H, d = t.shape
        wide = torch.zeros(T, H * d + odd, dtype=BF, device=dev)
        wide[:, int(odd):] = t.reshape(T, -1).to(dev)
        return wide[:, int(odd):].unflatten(1, (H, d))
    out, fin = decay_prefill(place(q), place(k), place(v), ld.to(dev), cu.to(dev), init.to(dev))
    ref.close("out", out, ro)
    ref.close("state", fin, rf)


@pytest.mark.parametrize("dk,dv", [(32, 64), (64, 128)])
def test_timeout(dk, dv):
    dev = need_gpu()
    args = [t.to(dev) for t in _inputs([90, 40], 2, dk, dv, 4)]
    want = decay_prefill(*args)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    kda.testing_expire_next_wait(kda.KDA_TESTING_DECAY)
    decay_prefill(*args, status=status)
    assert check_device_status(status) == kda.KDA_ERR_DEVICE_TIMEOUT
    status.zero_()
    got = decay_prefill(*args, status=status)
    assert check_device_status(status) == kda.KDA_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want))
