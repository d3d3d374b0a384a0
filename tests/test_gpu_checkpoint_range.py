"""The backward from a checkpoint over the range of the norm, against fp64
autograd (tests/_train_ref.py): streams far from 1, rows of zeros, eps near or
at zero. The statistic is a mean, finite wherever a thread's own squares
are, and the gradients with it; beyond that they are NaN, never silently zero.

Bars: C roundings (2^-24) on the absolute values that enter a result, plus half
a step of its type. C = 192: the second term of P_i = <dh, H_i> multiplies the
sums u h and h H_i by r^2, each sum a chain of at most n + 1 terms mixed into
h, 3 slices of 8 columns, 5 exchanges in a warp and 10 warps (48), r half of
another such sum's and 2 of its own (26).
"""
from __future__ import annotations

import pytest
import torch

from tests import _train_ref as R

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
C = 192


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


# both kernels: rows read directly (short, or n > 4) and rows copied whole
SHAPES = [(37, 4, 1024, "bf16"), (21, 8, 520, "bf16"), (40, 2, 1000, "f32"), (160, 4, 7168, "bf16"),
          (155, 2, 2592, "f32"), (151, 1, 5136, "bf16")]


def _check(hc, H, y, eps, dx, dHo, seed):
    T, n, d = H.shape
    cH, cy = hc.checkpoint_pack(H.cuda()), hc.checkpoint_pack(y.cuda())
    A = (torch.eye(n) + _normal(seed, T, n, n, std=0.3)).cuda()
    b, a = _normal(seed + 1, T, n, mean=1.0, std=0.2).cuda(), (_normal(seed + 2, T, n, std=0.3) + 1.0 / n).cuda()
    g = (_normal(seed + 3, d, std=0.3) + 1).cuda()
    got = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, None if dHo is None else dHo.cuda(), dx.cuda(),
                                                 eps=eps)
    kept = [hc.checkpoint_unpack(c, torch.float32).double().cpu() for c in (cH, cy)]
    p = [t.double().cpu() for t in (A, b, a, g)]
    eps = float(torch.tensor(eps, dtype=torch.float32))
    args = (*kept, *p, eps, dHo, dx, 0, 0, 0)
    ref, bound = R.step_grads(*args), R.step_bounds(*args)
    for k in ref:
        assert ref[k].isfinite().all()
        step = R.HALF_STEP[dx.dtype] if k in ("dH", "dy") else R.U
        R.check_as(k, got[k], ref[k], bound[k], C, step)


@pytest.mark.parametrize("scale,eps,up", [(1e15, 1e-6, 1.0), (1e12, 1e-6, 1.0), (1e-14, 0.0, 1.0), (1e-9, 1e-30, 1.0),
                                          (1e17, 1e-6, 1e-5), (1e15, 0.0, 1e15)])
@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_streams_far_from_one(hc, T, n, d, dt, scale, eps, up):
    """Streams of size `scale` and gradients of size `up` arriving: with the
    norm's own dx alone, which the streams' size hides no part of, and with
    dH' of the size that dx has in dH."""
    H, y = _normal(50, T, n, d) * scale, _normal(51, T, d) * scale
    dx = (_normal(52, T, d) * up).to(DT[dt])
    _check(hc, H, y, eps, dx, None, 53)
    _check(hc, H, y, eps, dx, (_normal(57, T, n, d) * (up / scale)).to(DT[dt]), 53)


@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_rows_of_zeros(hc, T, n, d, dt):
    """A token of zeros has the gradient dh = u / sqrt(eps) and no gradient of
    its weights, however small eps is."""
    H, y = _normal(60, T, n, d), _normal(61, T, d)
    H[::5], y[::5] = 0.0, 0.0
    dx = _normal(62, T, d).to(DT[dt])
    for eps in (1e-30, 1e-12, 1e-6):
        _check(hc, H, y, eps, dx, None, 63)


@pytest.mark.parametrize("T,n,d,dt", SHAPES)
def test_rows_beyond_the_range(hc, T, n, d, dt):
    """|h| above 1e19: no norm, so NaN in everything the norm enters, in these
    tokens only."""
    H, y = _normal(70, T, n, d), _normal(71, T, d)
    H[3], H[7, 0] = H[3] * 1e22, H[7, 0] * 1e25
    cH, cy = hc.checkpoint_pack(H.cuda()), hc.checkpoint_pack(y.cuda())
    A, b, a = torch.eye(n).cuda() + 0.25, torch.ones(n).cuda(), torch.full((n,), 0.5).cuda()
    dx, g = _normal(72, T, d).to(DT[dt]).cuda(), torch.ones(d).cuda()
    got = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, None, dx)
    rest = [t for t in range(T) if t not in (3, 7)]
    part = lambda c: hc.Checkpoint(c.codes.view(torch.uint8)[rest].view(torch.float8_e4m3fn), c.scales[rest])
    want = hc.write_then_read_backward_checkpoint(part(cH), part(cy), A, b, a, g, None, dx[rest])
    for k in ("dH", "dy", "dA", "db", "da"):
        assert got[k][3].isnan().all() and got[k][7].isnan().all(), k
        assert torch.equal(got[k][rest], want[k]), k
    assert got["dg"].isnan().all()
