"""kda_linear (projection with bias, activation and residual) against float64."""
import pytest
import torch

import layers_ref as ref
from gated_delta_rule_46_gb300 import KDAError, linear
from gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ACTS = ["none", "relu", "gelu", "silu", "sigmoid"]


def _inputs(M, N, K, bias, residual, odt, seed, ld=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, ld or K, generator=g).to(torch.bfloat16)
    w = (torch.randn(N, K, generator=g) / K ** 0.5).to(torch.bfloat16)
    b = 0.1 * torch.randn(N, generator=g) if bias else None
    r = torch.randn(M, N, generator=g).to(odt) if residual else None
    return x, w, b, r


def _run(M, N, K, bias, residual, act, odt, ld=None, seed=0):
    dev = need_gpu()
    x, w, b, r = _inputs(M, N, K, bias, residual, odt, seed, ld)
    xd = x.to(dev)[:, :K]
    got = linear(xd, w.to(dev), None if b is None else b.to(dev), None if r is None else r.to(dev), act=act,
                 out_dtype=odt)
    torch.cuda.synchronize()
    assert got.dtype == odt
    ref.close(f"{M}x{N}x{K} {act}", got, ref.linear(x[:, :K], w, b, r, act))


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 33, 64, 65, 127, 128, 129, 200, 256, 257, 384, 700])
@pytest.mark.parametrize("N,K", [(8, 8), (128, 64), (136, 72), (520, 1032), (1000, 512)])
def test_row_counts(M, N, K):
    _run(M, N, K, True, True, "silu", torch.bfloat16, seed=M)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_epilogues(act, bias, residual, odt):
    _run(40, 264, 256, bias, residual, act, odt, seed=1)
    _run(300, 264, 256, bias, residual, act, odt, seed=2)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 7), (17, 33, 100), (130, 131, 129), (64, 9, 2050), (5, 129, 64),
                                   (300, 1, 64), (260, 515, 128), (1, 4097, 96), (513, 77, 520)])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
def test_odd_sizes(M, N, K, odt):
    _run(M, N, K, True, True, "gelu", odt, seed=3)


@pytest.mark.parametrize("M", [5, 48, 400])
@pytest.mark.parametrize("ld", [520, 517, 544])
def test_row_stride(M, ld):
    """x as a slice of wider rows, 16-byte aligned and not."""
    _run(M, 192, 512, True, False, "none", torch.bfloat16, ld=ld, seed=4)


@pytest.mark.parametrize("M,N,K", [(64, 512, 8192), (1024, 640, 4096), (2500, 2056, 1024)])
def test_long_sums_and_many_tiles(M, N, K):
    _run(M, N, K, True, False, "none", torch.float32, seed=5)
    _run(M, N, K, False, True, "relu", torch.bfloat16, seed=6)


@pytest.mark.parametrize("M", [6, 64, 300])
def test_residual_in_place(M):
    dev = need_gpu()
    x, w, b, r = _inputs(M, 256, 512, True, True, torch.bfloat16, 7)
    buf = r.to(dev)
    got = linear(x.to(dev), w.to(dev), b.to(dev), residual=buf, out=buf)
    assert got is buf
    ref.close("in place", buf, ref.linear(x, w, b, r, "none"))


@pytest.mark.parametrize("M", [4, 100, 260])
def test_rows_are_independent(M):
    """NaN and infinity in one row of x stay in that row; a weight row's in its column."""
    dev = need_gpu()
    x, w, b, r = _inputs(M, 136, 256, False, False, torch.bfloat16, 8)
    clean = linear(x.to(dev), w.to(dev))
    x2, w2 = x.clone(), w.clone()
    x2[1, 5] = float("nan")
    x2[3, 9] = float("inf")
    w2[7, 0] = float("nan")
    got = linear(x2.to(dev), w2.to(dev))
    rows = [i for i in range(M) if i not in (1, 3)]
    cols = [i for i in range(136) if i != 7]
    assert torch.equal(got[rows][:, cols], clean[rows][:, cols])
    assert torch.isnan(got[1]).all() and torch.isnan(got[:, 7]).all()
    assert not torch.isfinite(got[3]).any()


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu"])
def test_activation_limits(act):
    """Sums far out on both sides: no NaN from the exponential's overflow."""
    dev = need_gpu()
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    x[:, 0] = torch.tensor([-300.0, -40.0, 40.0, 300.0])
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    w[:, 0] = 1
    got = linear(x.to(dev), w.to(dev), act=act, out_dtype=torch.float32).cpu()
    want = ref.linear(x, w, None, None, act)
    assert torch.isfinite(got).all()
    assert float((got.double() - want).abs().max()) <= 300 * 2.0 ** -20


def test_empty_and_deterministic():
    dev = need_gpu()
    x, w, b, _ = _inputs(70, 264, 4096, True, False, torch.bfloat16, 9)
    xd, wd, bd = x.to(dev), w.to(dev), b.to(dev)
    assert linear(xd[:0], wd, bd).shape == (0, 264)
    assert linear(xd, wd[:0]).shape == (70, 0)
    a = linear(xd, wd, bd)
    for _ in range(3):
        assert torch.equal(a, linear(xd, wd, bd))


def test_other_stream():
    dev = need_gpu()
    x, w, b, r = _inputs(200, 512, 1024, True, True, torch.bfloat16, 10)
    xd, wd, bd, rd = x.to(dev), w.to(dev), b.to(dev), r.to(dev)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = linear(xd, wd, bd, rd, act="silu", stream=s)
    s.synchronize()
    ref.close("side stream", got, ref.linear(x, w, b, r, "silu"))


def test_refusals():
    dev = need_gpu()
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(8, 16, dtype=torch.bfloat16, device=dev)
    with pytest.raises(TypeError):
        linear(x.float(), w)
    with pytest.raises(TypeError):
        linear(x, w.float())
    with pytest.raises(ValueError):
        linear(x, w[:, :8].contiguous())
    with pytest.raises(ValueError):
        linear(x, w[:, ::2])
    with pytest.raises(ValueError):
        linear(x.t(), w)
    with pytest.raises(ValueError):
        linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        linear(x, w, bias=torch.zeros(9, device=dev))
    with pytest.raises(TypeError):
        linear(x, w, residual=torch.zeros(4, 8, device=dev))
    with pytest.raises(TypeError):
        linear(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        linear(x, w.cpu())
    with pytest.raises(KDAError):
        linear(x[:, :0], w[:, :0].contiguous())


@pytest.mark.parametrize("M,N,K", [(700, 2056, 200), (1024, 1032, 136), (260, 6000, 64), (200, 10240, 264), (2304, 2304, 72)])
@pytest.mark.parametrize("odt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("residual", [False, True])
def test_pair_tiles(M, N, K, odt, residual):
    """Sizes that the CTA-pair kernel takes, both tile widths, edges in every direction."""
    _run(M, N, K, True, residual, "gelu", odt, seed=11)
