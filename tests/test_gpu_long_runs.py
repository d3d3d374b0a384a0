"""Training calls with several tokens a CTA and several batches of parameters,
where sums run on from token to token: the kernels that read rows directly (the
layer-norm backward of rows that are too wide for the staged form, or of codes
that do not start on 16 bytes; the backward from a checkpoint beyond four
streams and of short rows), against fp64 definitions (tests/_train_ref.py).

Bars: C roundings (2^-24) on the absolute values that enter a result plus half
a step of its type. Layer norm, C = 96: 28 slices a thread of 8 columns at
most, 5 exchanges and 8 warps for the statistics (41, and as much again in the
products they enter), one add a token of a CTA for dg and dbeta (at most 8
here). Checkpoint, C = 192: as in test_gpu_checkpoint_range.py, n + 1 at most 9
and one add a token; Sinkhorn adds 2 K (n + 1) and the softmax 2 n + 8, and
gradients of logits have the bar of the full-precision backward's tests, 2e-4
of the largest.

The chains of fp32 roundings as the kernels have them, which the bars of 64 and
32 of the other training tests stand for as well. Backward from a checkpoint:
h n + 1; a thread's sum 24 (three slices of 8 in turn) or 5 and an add a slice
(16 at the widest); 1 for the division by d; 5 exchanges; 6 or 8 for the warps:
at most 36 and 44 with h. Layer norm: a thread's squares 32 (8 slices), 5
exchanges, 5 for the warps, of which the inverse norm takes half; the mean's
own rounding is carried along and costs nothing. dg and dbeta: one add a token
of a CTA before the rows of partial sums are added in fp64.
"""
from __future__ import annotations

import pytest
import torch

from tests import _train_ref as R

pytestmark = pytest.mark.gpu
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


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
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


@pytest.mark.parametrize("T,n,d,dt,read,packed", [
    (1000, 4, 7168, "bf16", "logits", False), (700, 1, 8192, "bf16", "none", False),
    (1500, 3, 1032, "bf16", "token", True), (700, 2, 4096, "f32", "weights", False),
    (1201, 8, 4096, "bf16", "logits", False), (800, 2, 8200, "bf16", "logits", True),
    (2500, 1, 1004, "f32", "none", True), (640, 4, 8192, "bf16", "none4", False)])
def test_layernorm_backward(hc, T, n, d, dt, read, packed):
    H = _normal(1, T, n, d, mean=0.3).to(DT[dt])
    a = {"none": None, "none4": _normal(2, n), "weights": _normal(2, n, std=0.4) + 0.5,
         "token": _normal(2, T, n) + 0.5, "logits": _normal(2, T, n)}[read]
    soft = int(read in ("logits", "none4"))
    g, dx = _normal(3, d, std=0.3) + 1, _normal(4, T, d).to(DT[dt])
    src = hc.checkpoint_pack(H) if packed else H
    vals = hc.checkpoint_unpack(src, torch.float32) if packed else H
    got = hc.read_layernorm_backward(src, a, g, dx, eps=EPS, read=soft)
    again = hc.read_layernorm_backward(src, a, g, dx, eps=EPS, read=soft)
    for k in got:
        assert got[k] is None and again[k] is None or torch.equal(got[k], again[k]), k
    d64 = lambda t: None if t is None else t.double()
    ref = R.layernorm_grads(vals.double(), d64(a), d64(g), EPS, dx.double(), soft)
    bound = R.layernorm_bounds(vals.double(), d64(a), d64(g), None, EPS, dx.double(), soft)
    for k in ref:
        R.check_as(k, got[k], ref[k], bound[k], 96, R.HALF_STEP[dx.dtype] if k == "dH" else R.U)


@pytest.mark.parametrize("T,n,d,dt,logits,shared", [
    (700, 5, 2056, "bf16", True, False), (900, 6, 1024, "bf16", False, True), (650, 7, 520, "bf16", True, False),
    (1100, 8, 1024, "bf16", True, False), (620, 5, 1000, "f32", True, True), (640, 6, 516, "f32", False, False),
    (610, 7, 1024, "f32", True, False), (600, 8, 2048, "f32", False, True), (3000, 4, 264, "bf16", True, False),
    (1300, 3, 1544, "bf16", False, False), (5000, 1, 72, "f32", False, False), (600, 8, 4096, "bf16", True, False)])
def test_checkpoint_backward(hc, T, n, d, dt, logits, shared):
    cH, cy = hc.checkpoint_pack(_normal(11, T, n, d)), hc.checkpoint_pack(_normal(12, T, d))
    lead, K = () if shared else (T,), 20
    A = _normal(13, *lead, n, n) if logits else torch.eye(n, device="cuda") + _normal(13, *lead, n, n, std=0.3)
    a = _normal(14, *lead, n) if logits else _normal(14, *lead, n, std=0.3) + 1.0 / n
    b, g = _normal(15, *lead, n, mean=1.0, std=0.2), _normal(16, d, std=0.3) + 1
    dHo, dx = _normal(17, T, n, d).to(DT[dt]), _normal(18, T, d).to(DT[dt])
    kw = dict(eps=EPS, mix=int(logits), K=K if logits else 0, read=int(logits))
    got = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    again = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    for k in got:
        assert torch.equal(got[k], again[k]), k
    vH, vy = (hc.checkpoint_unpack(c, torch.float32).double() for c in (cH, cy))
    args = (vH, vy, A.double(), b.double(), a.double(), g.double(), EPS, dHo.double(), dx.double(), kw["mix"], kw["K"],
            kw["read"])
    ref, bound = R.step_grads(*args), R.step_bounds(*args)
    C = 192 + (2 * K * (n + 1) + 2 * n + 8 if logits else 0)
    for k in ref:
        if logits and k in ("dA", "da"):
            off = (got[k].double() - ref[k]).abs().max()
            assert off <= 2e-4 * ref[k].abs().max() + C * R.U * bound[k].max(), (k, float(off))
        else:
            R.check_as(k, got[k], ref[k], bound[k], C, R.HALF_STEP[dx.dtype] if k in ("dH", "dy") else R.U)
