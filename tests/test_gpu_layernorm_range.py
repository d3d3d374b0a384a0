"""Layer-norm reads over the range of the norm, forward and backward, against
fp64 definitions (tests/_train_ref.py): rows far from 1 in size, rows of one
value, eps near or at zero. The norm is taken from a mean of squares, finite
wherever a thread's own squares are; beyond that a row is NaN, never silently
beta with no gradient.

Bars: those of test_gpu_layernorm_far_mean.py, C = 64 roundings on sums of
absolute values, with s (sum |a_i H_i| + |mean|) for z.
"""
from __future__ import annotations

import pytest
import torch

from tests import _train_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
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


# rows the staged backward takes, and rows the direct one does
SHAPES = [(160, 1, 7168, "bf16"), (40, 4, 1024, "bf16"), (33, 2, 3584, "f32"), (155, 4, 7168, "bf16"),
          (20, 1, 8192, "bf16"), (21, 3, 8200, "f32"), (30, 8, 4096, "bf16")]


def _inputs(T, n, d, dt, scale):
    H = (_normal(80, T, n, d, mean=0.5) * scale).to(DT[dt])
    return H, _normal(81, T, n, std=0.3) + 0.5, _normal(82, d, std=0.3) + 1, _normal(83, d, std=0.5)


def _check(hc, H, a, g, beta, dx, eps, sums=True):
    dev = [t.cuda() for t in (H, a, g, beta, dx)]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    d64 = [t.double() for t in (H, a, g, beta, dx)]
    bound = R.layernorm_bounds(*d64[:4], eps, d64[4], 0)
    x = hc.read_layernorm(*dev[:4], eps=eps)
    R.check_as("x", x, R.layernorm(*d64[:4], eps, 0), bound["x"], C, R.HALF_STEP[H.dtype])
    got = hc.read_layernorm_backward(*dev[:3], dev[4], eps=eps)
    ref = R.layernorm_grads(*d64[:3], eps, d64[4], 0)
    for k in ref if sums else ("dH", "da"):
        R.check_as(k, got[k], ref[k], bound[k], C, R.HALF_STEP[H.dtype] if k == "dH" else R.U)


@pytest.mark.parametrize("scale,eps,up", [(1e15, 1e-6, 1.0), (1.5e17, 1e-6, 1.0), (1e17, 1e-6, 1e17), (1e-14, 0.0, 1.0),
                                          (1e-9, 1e-30, 1.0)])
@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_rows_far_from_one(hc, T, n, d, dt, scale, eps, up):
    H, a, g, beta = _inputs(T, n, d, dt, scale)
    _check(hc, H, a, g, beta, (_normal(84, T, d) * up).to(DT[dt]), eps)


@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_rows_of_one_value(hc, T, n, d, dt):
    """No deviation: x = beta and dh = (u - mean u) / sqrt(eps), however small
    eps is."""
    H, a, g, beta = _inputs(T, n, d, dt, 1.0)
    H[::3] = 0.0
    for eps in (1e-30, 1e-12):
        _check(hc, H, a, g, beta, _normal(85, T, d).to(DT[dt]), eps)


@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_rows_beyond_the_range(hc, T, n, d, dt):
    """Deviations above 1e19: NaN, in these tokens only."""
    H, a, g, beta = (t.cuda() for t in _inputs(T, n, d, dt, 1.0))
    H[3], H[7, 0] = H[3] * 1e22, H[7, 0] * 1e25
    dx = _normal(86, T, d).to(DT[dt]).cuda()
    x, got = hc.read_layernorm(H, a, g, beta), hc.read_layernorm_backward(H, a, g, dx)
    rest = [t for t in range(T) if t not in (3, 7)]
    want = hc.read_layernorm_backward(H[rest], a[rest], g, dx[rest])
    assert x[3].isnan().all() and x[7].isnan().all()
    assert torch.equal(x[rest], hc.read_layernorm(H[rest], a[rest], g, beta))
    for k in ("dH", "da"):
        assert got[k][3].isnan().all() and got[k][7].isnan().all(), k
        assert torch.equal(got[k][rest], want[k]), k
    assert got["dg"].isnan().all() and got["dbeta"].isfinite().all()
