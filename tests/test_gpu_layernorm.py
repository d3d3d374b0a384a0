"""The layer-norm read and its gradients on the GPU against fp64 definitions
(tests/_train_ref.py).

Bars: C roundings (2^-24) on the absolute values that enter a result plus half
a step of its type. C = 32 forward: up to 8 in the mix, 4 for the read softmax
and its exp, 6 from h to x, and the moments' own (a thread sums its deviations
from a pivot, at most twice the row's, over its slices: 2 * 8). C = 64
backward, whose sums run over a thread's slices (28 at the widest row here),
a warp and a CTA's tokens. A rounding of h or of the mean counts by what it
does to the normalised value, s (sum |a_i H_i| + |mean|).
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
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std + mean


def _inputs(seed, T, n, d, dt, read, offset=0.3):
    H = _normal(seed, T, n, d, mean=offset).to(DT[dt]).cuda()
    a = {"none": None, "weights": _normal(seed + 1, n, std=0.4) + 0.5, "token": _normal(seed + 1, T, n) + 0.5,
         "logits": _normal(seed + 1, T, n)}[read]
    a = a if a is None else a.cuda()
    g, beta = (_normal(seed + 2, d, std=0.3) + 1).cuda(), _normal(seed + 3, d, std=0.5).cuda()
    dx = _normal(seed + 4, T, d).to(DT[dt]).cuda()
    return H, a, g, beta, dx, int(read == "logits")


CASES = [
    (1, 4, 7168, "bf16", "logits"), (1, 1, 7168, "bf16", "none"), (64, 4, 4096, "bf16", "token"),
    (37, 2, 1000, "f32", "weights"), (300, 1, 7168, "bf16", "none"), (51, 1, 1032, "f32", "none"),
    (33, 8, 520, "bf16", "logits"), (20, 3, 264, "bf16", "weights"), (7, 4, 8, "bf16", "logits"),
    (7, 2, 4, "f32", "token"), (129, 6, 776, "bf16", "token"), (1200, 4, 1024, "bf16", "logits"),
    (41, 5, 1544, "f32", "logits"), (26, 7, 2056, "bf16", "logits"), (2000, 1, 512, "f32", "none"),
    (5, 2, 32768, "bf16", "logits"), (5, 1, 16384, "f32", "none"), (3, 8, 16384, "bf16", "weights"),
    (900, 1, 4096, "bf16", "none"), (650, 2, 7168, "bf16", "token"),
]


def _cpu(*ts):
    return [None if t is None else t.double().cpu() for t in ts]


@pytest.mark.parametrize("T,n,d,dt,read", CASES)
def test_forward(hc, T, n, d, dt, read):
    H, a, g, beta, _, soft = _inputs(100 + T + n, T, n, d, dt, read)
    for gg, bb in ((g, beta), (None, beta), (g, None), (None, None)):
        x = hc.read_layernorm(H, a, gg, bb, eps=EPS, read=soft)
        assert x.dtype == H.dtype and x.shape == (T, d)
        ref = R.layernorm(*_cpu(H, a, gg, bb), EPS, soft)
        bound = R.layernorm_bounds(*_cpu(H, a, gg, bb), EPS, None, soft)["x"]
        R.check_as("x", x, ref, bound, 32, R.HALF_STEP[H.dtype])


def _check_grads(got, H, a, g, dx, soft, sl=slice(None), sums=True):
    p = lambda t: t if t is None or t.dim() == 1 else t[sl]
    args = (*_cpu(H[sl], p(a), g), EPS, dx[sl].double().cpu(), soft)
    ref = R.layernorm_grads(*args)
    bound = R.layernorm_bounds(args[0], args[1], args[2], None, *args[3:])
    assert got["dH"].dtype == dx.dtype
    R.check_as("dH", got["dH"][sl], ref["dH"], bound["dH"], 64, R.HALF_STEP[dx.dtype])
    assert (got["da"] is None) == (a is None) and (got["dg"] is None) == (g is None)
    if a is not None:
        R.check_as("da", got["da"][sl], ref["da"], bound["da"], 64, R.U)
    if sums:
        if g is not None:
            R.check_as("dg", got["dg"], ref["dg"], bound["dg"], 64, R.U)
        R.check_as("dbeta", got["dbeta"], ref["dbeta"], bound["dbeta"], 64, R.U)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,n,d,dt,read", CASES)
def test_backward(hc, T, n, d, dt, read, packed):
    H, a, g, _, dx, soft = _inputs(200 + T + n, T, n, d, dt, read)
    src = hc.checkpoint_pack(H) if packed else H
    got = hc.read_layernorm_backward(src, a, g, dx, eps=EPS, read=soft)
    _check_grads(got, hc.checkpoint_unpack(src, torch.float32) if packed else H, a, g, dx, soft)


def test_backward_without_gain_or_sums(hc):
    H, a, g, _, dx, soft = _inputs(300, 70, 3, 1032, "bf16", "logits")
    full = hc.read_layernorm_backward(H, a, g, dx, read=soft)
    for kw in (dict(want_dg=False), dict(want_dbeta=False), dict(want_dg=False, want_dbeta=False)):
        got = hc.read_layernorm_backward(H, a, g, dx, read=soft, **kw)
        assert (got["dg"] is None) == ("want_dg" in kw) and (got["dbeta"] is None) == ("want_dbeta" in kw)
        for k in full:
            assert got[k] is None or torch.equal(got[k], full[k]), k
    _check_grads(hc.read_layernorm_backward(H, a, None, dx, read=soft), H, a, None, dx, soft)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_mean_far_from_zero(hc, dt):
    """A mean 200 times the deviation: the moments lose nothing to it beyond
    the rounding of h itself."""
    H, a, g, beta, dx, soft = _inputs(400, 40, 1, 7168, dt, "none", offset=200.0)
    x = hc.read_layernorm(H, a, g, beta, eps=EPS)
    ref = R.layernorm(*_cpu(H, a, g, beta), EPS, 0)
    # n = 1, weight 1: h is H itself, and h - mean rounds at its own size
    z = (ref - beta.double().cpu()).abs()
    bar = 32 * R.U * (z + beta.double().cpu().abs() + 1) + R.HALF_STEP[H.dtype] * ref.abs() * (1 + 2.0 ** -6)
    assert bool(((x.double().cpu() - ref).abs() <= bar).all())
    _check_grads(hc.read_layernorm_backward(H, a, g, dx), H, a, g, dx, 0)


def test_constant_rows_and_not_finite_rows(hc):
    """A constant row has x = beta and no gradient into H; a row with an
    infinity or NaN is NaN and leaves the others alone."""
    T, d = 30, 1024
    H, _, g, beta, dx, _ = _inputs(410, T, 1, d, "f32", "none")
    H[4] = 3.25
    H[6, 0, 100] = float("inf")
    H[8, 0, 0] = float("nan")
    x = hc.read_layernorm(H, None, g, beta)
    assert torch.equal(x[4], beta)
    assert x[6].isnan().all() and x[8].isnan().all()
    keep = [t for t in range(T) if t not in (6, 8)]
    assert torch.equal(x[keep], hc.read_layernorm(H[keep].contiguous(), None, g, beta))
    got = hc.read_layernorm_backward(H, None, g, dx)
    same = hc.read_layernorm_backward(H[keep].contiguous(), None, g, dx[keep].contiguous())
    assert torch.equal(got["dH"][keep], same["dH"])
    assert got["dH"][6].isnan().all() and got["dH"][8].isnan().all()
    assert got["dH"][4].isfinite().all()


def test_gradients_against_differences(hc):
    """Central differences of the fp64 read along random directions."""
    T, n, d = 7, 3, 96
    H, a, g, beta, dx, soft = _inputs(420, T, n, d, "f32", "logits")
    got = hc.read_layernorm_backward(H, a, g, dx, read=soft)
    v = dict(zip(("dH", "da", "dg", "dbeta"), _cpu(H, a, g, beta)))
    for i, k in enumerate(v):
        e, h = _normal(430 + i, *v[k].shape).double(), 1e-4
        at = lambda s: float((R.layernorm(*(dict(v, **{k: v[k] + s * e})[q] for q in ("dH", "da", "dg", "dbeta")),
                                          EPS, soft) * dx.double().cpu()).sum())
        want = (at(h) - at(-h)) / (2 * h)
        terms = got[k].double().cpu() * e
        # the roundings on the terms, 16 times their sum where the two means are taken out
        assert abs(float(terms.sum()) - want) <= 64 * 16 * R.U * float(terms.abs().sum()) + 1e-6, k


def test_streams_graphs_and_in_place_norm(hc):
    T, n, d = 500, 2, 4096
    H, a, g, beta, dx, soft = _inputs(440, T, n, d, "bf16", "logits")
    H2, a2, _, _, dx2, _ = _inputs(450, T, n, d, "bf16", "logits")
    x, gr = hc.read_layernorm(H, a, g, beta, read=soft), hc.read_layernorm_backward(H, a, g, dx, read=soft)
    x2, gr2 = hc.read_layernorm(H2, a2, g, beta, read=soft), hc.read_layernorm_backward(H2, a2, g, dx2, read=soft)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(s1):
        y1 = hc.read_layernorm_backward(H, a, g, dx, read=soft)
    with torch.cuda.stream(s2):
        y2 = hc.read_layernorm_backward(H2, a2, g, dx2, read=soft)
    torch.cuda.synchronize()
    for k in gr:
        assert torch.equal(y1[k], gr[k]) and torch.equal(y2[k], gr2[k]), k
    Hs, as_, dxs = H.clone(), a.clone(), dx.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        xs = hc.read_layernorm(Hs, as_, g, beta, read=soft)
        ys = hc.read_layernorm_backward(Hs, as_, g, dxs, read=soft)
    for (h, w, u), rx, rg in (((H2, a2, dx2), x2, gr2), ((H, a, dx), x, gr)):
        Hs.copy_(h)
        as_.copy_(w)
        dxs.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(xs, rx)
        for k in rg:
            assert torch.equal(ys[k], rg[k]), k


def test_past_32_bit_offsets(hc):
    T, n, d = 75100, 4, 7168
    gen = torch.Generator(device="cuda").manual_seed(9)
    H = torch.empty(T, n, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    dx = torch.empty(T, d, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    a, g = _normal(1, T, n).cuda(), torch.ones(d, device="cuda")
    x = hc.read_layernorm(H, a, g, None, read=1)
    got = hc.read_layernorm_backward(H, a, g, dx, read=1)
    sl = slice(T - 3, T)
    ref = R.layernorm(*_cpu(H[sl], a[sl], g, None), EPS, 1)
    R.check_as("x", x[sl], ref, R.layernorm_bounds(*_cpu(H[sl], a[sl], g, None), EPS, None, 1)["x"], 32, 2.0 ** -8)
    _check_grads(got, H, a, g, dx, 1, sl=sl, sums=False)


def test_neighbours_stay(hc):
    """Rows before and after an output are not written."""
    T, n, d = 21, 3, 1032
    H, a, g, beta, _, soft = _inputs(460, T, n, d, "bf16", "logits")
    buf = torch.full((T + 2, d), 7.0, dtype=torch.bfloat16, device="cuda")
    hc.read_layernorm(H, a, g, beta, read=soft, x=buf[1:-1])
    assert (buf[0] == 7).all() and (buf[-1] == 7).all()
    assert torch.equal(buf[1:-1], hc.read_layernorm(H, a, g, beta, read=soft))


def test_refusals_on_the_gpu(hc):
    T, n, d = 8, 4, 64
    H = torch.zeros(T, n, d, device="cuda", dtype=torch.bfloat16)
    dx = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    a, g = torch.ones(n, device="cuda"), torch.ones(d, device="cuda")
    for call, err in [
        (lambda: hc.read_layernorm(H, None, g), ValueError),
        (lambda: hc.read_layernorm(H.half(), a, g), ValueError),
        (lambda: hc.read_layernorm(H, a, g[:32]), ValueError),
        (lambda: hc.read_layernorm(H, a, g, beta=g.bfloat16()), ValueError),
        (lambda: hc.read_layernorm(H, a[:3], g), ValueError),
        (lambda: hc.read_layernorm_backward(H, a, g, dx.float()), ValueError),
        (lambda: hc.read_layernorm_backward(H, a, g, dx[:4]), ValueError),
        (lambda: hc.read_layernorm_backward(H, a.cpu(), g, dx), ValueError),
    ]:
        with pytest.raises(err):
            call()
    for call, status in [
        (lambda: hc.read_layernorm(H, a, g, x=H.view(-1)[:T * d].view(T, d)), hc.HC_ERR_ALIAS),
        (lambda: hc.read_layernorm(H, a, g, eps=-1.0), hc.HC_ERR_INVALID_ARG),
        (lambda: hc.read_layernorm(H, a, g, read=5), hc.HC_ERR_INVALID_ARG),
        (lambda: hc.read_layernorm_backward(H, a, g, dx, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")),
         hc.HC_ERR_INVALID_ARG),
        (lambda: hc.read_layernorm(torch.zeros(2, 1, 12, device="cuda", dtype=torch.bfloat16), None),
         hc.HC_ERR_UNSUPPORTED),
    ]:
        with pytest.raises(hc.HCError) as e:
            call()
        assert e.value.status == status
    assert hc.read_layernorm(H[:0], a, g).shape == (0, d)
    out = hc.read_layernorm_backward(H[:0], a, g, dx[:0])
    assert out["dH"].shape == (0, n, d) and (out["dg"] == 0).all() and (out["dbeta"] == 0).all()
