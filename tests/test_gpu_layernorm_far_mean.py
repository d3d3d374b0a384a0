"""Layer-norm reads whose mean is thousands of deviations from zero, forward
and backward, whichever kernel the width selects, against fp64 definitions.

With one stream and no weights h is H itself, a number of fp32, and h - mean
rounds at its own size: the normalised value z is then off by roundings of
|z| + 1 (its moments are sums of deviations over a thread's columns, a warp and
the warps), whatever the mean is. Bars: C = 64 roundings on sums of absolute
values in which |z| + 1 stands for z: at most 28 adds in a thread, 5 in a warp,
14 warps, the difference of the means and four products.
"""
from __future__ import annotations

import pytest
import torch

from tests import _train_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6
C = 64


@pytest.fixture(scope="module")
def hc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hyper_connections_stream_b200 import build
    build.build()
    import hyper_connections_stream_b200._lib as L
    L.lib()
    yield L
    torch.cuda.synchronize()
    assert L.device_fault() == 0


def _normal(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std + mean


@pytest.mark.parametrize("mean", [2000.0, -20000.0, 300000.0])
@pytest.mark.parametrize("T,d", [(40, 2048), (600, 512), (300, 3584), (9, 36), (300, 4096), (3, 16384)])
def test_one_stream(hc, T, d, mean):
    H = _normal(70, T, 1, d, mean=mean).cuda()
    g, beta = (_normal(71, d, std=0.3) + 1).cuda(), _normal(72, d, std=0.5).cuda()
    dx = _normal(73, T, d).cuda()
    Hd, gd, bd, u = H.double().cpu(), g.double().cpu(), beta.double().cpu(), dx.double().cpu()
    h = Hd[:, 0] - Hd[:, 0].mean(-1, keepdim=True)
    s = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    z = (h * s).abs() + 1.0

    x = hc.read_layernorm(H, None, g, beta, eps=EPS)
    R.check_as("x", x, R.layernorm(Hd, None, gd, bd, EPS, 0), z * gd.abs() + bd.abs(), C, R.U)

    got = hc.read_layernorm_backward(H, None, g, dx, eps=EPS)
    ref = R.layernorm_grads(Hd, None, gd, EPS, u, 0)
    ua = u.abs() * gd.abs()
    dh = s * (ua + ua.mean(-1, keepdim=True) + z * (ua * z).mean(-1, keepdim=True))
    R.check_as("dH", got["dH"], ref["dH"], dh[:, None], C, R.U)
    R.check_as("dg", got["dg"], ref["dg"], (u.abs() * z).sum(0), C, R.U)
    R.check_as("dbeta", got["dbeta"], ref["dbeta"], u.abs().sum(0), C, R.U)


def test_one_stream_bf16(hc):
    """The same with rows of bf16: a mean of 96 deviations, where their step is
    half a deviation; both outputs rounded once."""
    T, d = 400, 7168
    H = _normal(75, T, 1, d, mean=96.0).bfloat16().cuda()
    g, dx = (_normal(76, d, std=0.3) + 1).cuda(), _normal(77, T, d).bfloat16().cuda()
    Hd, gd, u = H.double().cpu(), g.double().cpu(), dx.double().cpu()
    h = Hd[:, 0] - Hd[:, 0].mean(-1, keepdim=True)
    s = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    z, ua = (h * s).abs() + 1.0, u.abs() * gd.abs()
    got, ref = hc.read_layernorm_backward(H, None, g, dx, eps=EPS), R.layernorm_grads(Hd, None, gd, EPS, u, 0)
    dh = s * (ua + ua.mean(-1, keepdim=True) + z * (ua * z).mean(-1, keepdim=True))
    R.check_as("dH", got["dH"], ref["dH"], dh[:, None], C, R.HALF_STEP[torch.bfloat16])
    R.check_as("dg", got["dg"], ref["dg"], (u.abs() * z).sum(0), C, R.U)


def test_streams_of_one_mean(hc):
    """Streams that are one row and its double, so that their mix (a half and a
    quarter) is exact, far from zero."""
    T, d = 200, 1024
    row = _normal(78, T, d, mean=20000.0)
    H, a = torch.stack([row, 2 * row], 1).cuda(), torch.tensor([0.5, 0.25]).cuda()
    g, dx = (_normal(79, d, std=0.3) + 1).cuda(), _normal(80, T, d).cuda()
    gd, u = g.double().cpu(), dx.double().cpu()
    h = row.double() - row.double().mean(-1, keepdim=True)
    s = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
    z, ua = (h * s).abs() + 1.0, u.abs() * gd.abs()
    got = hc.read_layernorm_backward(H, a, g, dx, eps=EPS)
    ref = R.layernorm_grads(H.double().cpu(), a.double().cpu(), gd, EPS, u, 0)
    dh = s * (ua + ua.mean(-1, keepdim=True) + z * (ua * z).mean(-1, keepdim=True))
    R.check_as("dH", got["dH"], ref["dH"], a.double().cpu()[:, None] * dh[:, None], C, R.U)
    R.check_as("dg", got["dg"], ref["dg"], (u.abs() * z).sum(0), C, R.U)
