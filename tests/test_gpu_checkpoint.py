"""8-bit stream checkpoints on the GPU, the step that writes them and the
backward that reads them, against fp64 definitions (tests/_train_ref.py).

Codes and scales have one right value: they are compared exactly. Gradients:
C roundings (2^-24) on every absolute value that enters, plus half a step of
the output's own type. C counts the longest chain of fp32 roundings on a
term: up to n + 1 terms mixed into h, 4 in a slice, one add for each of a
thread's slices (28 at the widest row here), 5 in a warp, then fp64: 64 covers
them. Sinkhorn's 2 K passes add a division and n - 1 adds each: 2 K (n + 1)
roundings on A. The gradients of logits undo those passes, each a difference
of near-equal sums: 2e-4 of the largest magnitude, as in the tests of the
full-precision backward.
"""
from __future__ import annotations

import numpy as np
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


def _check_pack(hc, x):
    """x: CUDA tensor. Codes, scales and both unpackings against the search."""
    kept, e = R.pack_ref(x.double().cpu().numpy())
    d, nb = x.shape[-1], e.shape[-1]
    c = hc.checkpoint_pack(x)
    assert c.codes.shape == x.shape and c.codes.dtype == torch.float8_e4m3fn
    assert c.scales.shape == (*x.shape[:-1], hc.checkpoint_scale_stride(d))
    assert np.array_equal(c.scales[..., :nb].cpu().numpy(), e)
    codes = c.codes.view(torch.uint8).cpu().numpy()
    s = np.repeat(2.0 ** (e.astype(np.float64) - 127), 32, axis=-1)[..., :d]
    assert np.array_equal(R.e4m3_values()[codes] * s, kept, equal_nan=True)
    zero = (kept == 0) & (x.double().cpu().numpy() == 0)
    assert np.array_equal(np.signbit(R.e4m3_values()[codes][zero]), np.signbit(x.double().cpu().numpy()[zero]))
    for dt in (torch.float32, torch.bfloat16):
        if dt == torch.bfloat16 and d % 8:  # bf16 rows hold whole 16-byte vectors
            with pytest.raises(hc.HCError):
                hc.checkpoint_unpack(c, dt)
            continue
        v = hc.checkpoint_unpack(c, dt)
        assert v.dtype == dt and v.shape == x.shape
        want = torch.from_numpy(kept).to(torch.float32).to(dt).double().numpy()  # kept values fit fp32
        assert np.array_equal(v.double().cpu().numpy(), want, equal_nan=True)
    return c


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 8), (3, 40), (5, 1, 264), (2, 4, 1000), (37, 4, 1032), (9, 7168), (1, 32),
                                   (700, 96), (3, 2, 8200)])
def test_pack_matches_search(hc, dt, shape):
    x = _normal(11 + len(shape) + shape[-1], *shape) * torch.exp(_normal(5, shape[-1], std=2.0))
    _check_pack(hc, x.to(DT[dt]).cuda())


def test_pack_f32_row_of_four(hc):
    _check_pack(hc, _normal(3, 7, 4).cuda())
    _check_pack(hc, _normal(4, 7, 1004).cuda())


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_pack_range_and_special_values(hc, dt):
    """Blocks at the ends of the type's range, maxima next to 448 * 2^k, ties,
    zeros, and values that are not finite beside ones that are."""
    fi = torch.finfo(DT[dt])
    rows = []
    for k in range(-140, 121):
        for m in (448.0, 449.0, 452.0, 447.0, 256.0, 255.0, 511.0):
            v = np.ldexp(np.array([m, -m / 3, 0.0, -0.0, m * 2.0 ** -15, 17 / 32 * m, m / 7, 1e-3 * m] * 4), k)
            rows.append(np.clip(v, -fi.max, fi.max))
    rows.append(np.zeros(32))
    rows.append(np.full(32, fi.max))
    rows.append(np.full(32, -fi.tiny))
    rows.append(np.full(32, 2.0 ** -133))
    rows.append(np.r_[np.arange(16) / 16 + 1, -(np.arange(16) / 16 + 1)] * 256)      # ties between codes
    rows.append(np.r_[np.inf, -np.inf, np.nan, 3.0, np.arange(28) - 14.0])
    rows.append(np.full(32, np.inf))
    rows.append(np.full(32, np.nan))
    rows.append(np.r_[np.full(31, 1e-3), np.nan])
    x = torch.from_numpy(np.stack(rows)).float().to(DT[dt]).cuda()
    _check_pack(hc, x)
    _check_pack(hc, x.reshape(-1)[: x.numel() // 64 * 64].reshape(-1, 64)[:, :40].contiguous())


def test_pack_empty_and_untouched_neighbours(hc):
    """Zero rows; bytes around the outputs, and behind a row's last block, stay."""
    c = hc.checkpoint_pack(torch.empty(0, 4, 64, device="cuda"))
    assert hc.checkpoint_unpack(c).shape == (0, 4, 64)
    d, rows = 1032, 5
    ns = hc.checkpoint_scale_stride(d)
    q = torch.full(((rows + 2) * d + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    s = torch.full(((rows + 2) * ns,), 0xA5, dtype=torch.uint8, device="cuda")
    out = hc.Checkpoint(q[64:64 + rows * d].view(torch.float8_e4m3fn).view(rows, d), s[ns:ns + rows * ns].view(rows, ns))
    x = _normal(8, rows, d).bfloat16().cuda()
    hc.checkpoint_pack(x, out=out)
    assert (q[:64] == 0x5A).all() and (q[64 + rows * d:] == 0x5A).all()
    assert (s[:ns] == 0xA5).all() and (s[ns + rows * ns:] == 0xA5).all() and (out.scales[:, 33:] == 0xA5).all()
    v = torch.full((rows + 2, d), 7.0, device="cuda")
    hc.checkpoint_unpack(out, torch.float32, out=v[1:-1])
    assert (v[0] == 7).all() and (v[-1] == 7).all()
    assert torch.equal(v[1:-1], hc.checkpoint_unpack(hc.checkpoint_pack(x), torch.float32))


def test_pack_past_32_bit_offsets(hc):
    """More than 2^31 values: the first, a middle and the last rows."""
    rows, d = 300100, 7168
    x = torch.empty(rows, d, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x.normal_(generator=gen)
    c = hc.checkpoint_pack(x)
    v = hc.checkpoint_unpack(c)
    for r in (0, 1, rows // 2, rows - 2, rows - 1):
        kept, _ = R.pack_ref(x[r].double().cpu().numpy())
        assert np.array_equal(v[r].double().cpu().numpy(), kept)


# ---- the step that keeps a checkpoint ------------------------------------------------

def _params(seed, T, n, mix, read, shared):
    lead = () if shared else (T,)
    A = _normal(seed, *lead, n, n) if mix else torch.eye(n) + _normal(seed, *lead, n, n, std=0.3)
    a = _normal(seed + 1, *lead, n) if read else _normal(seed + 1, *lead, n, std=0.3) + 1.0 / n
    b = _normal(seed + 2, *lead, n, mean=1.0, std=0.2)
    return A.cuda(), b.cuda(), a.cuda()


@pytest.mark.parametrize("T,n,d,dt,logits,shared", [
    (1, 4, 7168, "bf16", True, False), (70, 4, 1032, "bf16", True, False), (33, 3, 1000, "f32", False, True),
    (600, 2, 2048, "bf16", True, False), (5, 1, 40, "f32", False, True), (41, 8, 520, "bf16", True, False),
    (900, 4, 7168, "bf16", True, False), (700, 4, 4096, "bf16", False, True), (300, 6, 1024, "f32", True, False),
    (2100, 8, 1024, "bf16", True, False), (1100, 5, 1544, "bf16", True, True), (2, 2, 32768, "bf16", False, True),
    (3, 2, 16384, "f32", False, True), (1500, 1, 7168, "bf16", False, True)])
def test_step_checkpoint_is_step_and_pack(hc, T, n, d, dt, logits, shared):
    """H' and x of write_then_read and the checkpoints of checkpoint_pack, bit
    for bit, out of place and in place."""
    H, y = _normal(21, T, n, d).to(DT[dt]).cuda(), _normal(22, T, d).to(DT[dt]).cuda()
    A, b, a = _params(23, T, n, logits, logits, shared)
    g = (_normal(26, d, std=0.2) + 1).cuda()
    kw = dict(eps=EPS, mix=int(logits), K=20 if logits else 0, read=int(logits))
    want = hc.write_then_read(H, y, A, b, a, g, **kw)
    wH, wy = hc.checkpoint_pack(H), hc.checkpoint_pack(y)
    nb = -(-d // 32)

    def same(c, w):
        assert torch.equal(c.codes.view(torch.uint8), w.codes.view(torch.uint8))
        assert torch.equal(c.scales[..., :nb], w.scales[..., :nb])

    Hn, x, cH, cy = hc.write_then_read_checkpoint(H, y, A, b, a, g, **kw)
    assert torch.equal(Hn, want[0]) and torch.equal(x, want[1])
    same(cH, wH)
    same(cy, wy)
    H2 = H.clone()
    Hn, x, cH, cy = hc.write_then_read_checkpoint(H2, y, A, b, a, g, out=H2, **kw)
    assert Hn is H2 and torch.equal(H2, want[0]) and torch.equal(x, want[1])
    same(cH, wH)
    same(cy, wy)


def test_step_checkpoint_keeps_infinities_to_their_token(hc):
    """A value that is not finite makes its own token's results what the plain
    step makes them, and is kept as NaN."""
    T, n, d = 40, 4, 1024
    H, y = _normal(31, T, n, d).bfloat16().cuda(), _normal(32, T, d).bfloat16().cuda()
    H[3, 1, 70] = float("inf")
    y[7, 1023] = float("nan")
    A, b, a = _params(33, T, n, True, True, False)
    kw = dict(mix=1, K=20, read=1)
    want = hc.write_then_read(H, y, A, b, a, **kw)
    Hn, x, cH, cy = hc.write_then_read_checkpoint(H, y, A, b, a, **kw)
    for got, w in ((Hn, want[0]), (x, want[1])):
        assert torch.equal(got.isnan(), w.isnan()) and torch.equal(got.nan_to_num(), w.nan_to_num())
    v = hc.checkpoint_unpack(cH, torch.float32)
    assert int(v.isnan().sum()) == 1 and bool(v[3, 1, 70].isnan())
    assert int(hc.checkpoint_unpack(cy, torch.float32).isnan().sum()) == 1


# ---- the backward from the checkpoint ---------------------------------------------------

def _backward_case(hc, T, n, d, dt, mix, read, shared, seed, with_dHout=True, gain=True, K=20):
    H, y = _normal(seed, T, n, d).cuda(), _normal(seed + 1, T, d).cuda()
    cH, cy = hc.checkpoint_pack(H), hc.checkpoint_pack(y)
    A, b, a = _params(seed + 2, T, n, mix, read, shared)
    g = (_normal(seed + 5, d, std=0.3) + 1).cuda() if gain else None
    dHo = _normal(seed + 6, T, n, d).to(DT[dt]).cuda() if with_dHout else None
    dx = _normal(seed + 7, T, d).to(DT[dt]).cuda()
    return cH, cy, A, b, a, g, dHo, dx, dict(eps=EPS, mix=int(mix), K=K if mix else 0, read=int(read))


def _check_backward(hc, got, cH, cy, A, b, a, g, dHo, dx, kw, sl=slice(None), sums=True):
    f = lambda t: None if t is None else t[sl].cpu()
    p = lambda t, dims: t.cpu() if t.dim() == dims else t[sl].cpu()
    kept = lambda c: hc.checkpoint_unpack(c, torch.float32)[sl].double().cpu()
    args = (kept(cH), kept(cy), p(A, 2).double(), p(b, 1).double(), p(a, 1).double(),
            None if g is None else g.cpu().double(), EPS, f(dHo), f(dx), kw["mix"], kw["K"], kw["read"])
    ref, bound = R.step_grads(*args), R.step_bounds(*args)
    n = A.shape[-1]
    C = 64 + (2 * kw["K"] * (n + 1) if kw["mix"] else 0) + (2 * n + 8 if kw["read"] else 0)
    step = R.HALF_STEP[dx.dtype]
    for k in ("dH", "dy"):
        assert got[k].dtype == dx.dtype
        R.check_as(k, got[k][sl], ref[k], bound[k], C, step)
    for k, logit in (("dA", kw["mix"]), ("db", 0), ("da", kw["read"])):
        if logit:
            off = (got[k][sl].double().cpu() - ref[k]).abs().max()
            assert off <= 2e-4 * ref[k].abs().max() + C * R.U * bound[k].max(), (k, float(off))
        else:
            R.check_as(k, got[k][sl], ref[k], bound[k], C, R.U)
    if sums:
        assert (got["dg"] is None) == (g is None)
        if g is not None:
            R.check_as("dg", got["dg"], ref["dg"], bound["dg"], C, R.U)


@pytest.mark.parametrize("T,n,d,dt,mix,read,shared", [
    (1, 4, 7168, "bf16", True, True, False),     # one token
    (37, 4, 1024, "f32", True, True, False),
    (64, 4, 2048, "bf16", True, True, False),
    (50, 2, 512, "f32", False, False, True),
    (33, 8, 512, "bf16", True, True, False),
    (33, 8, 1000, "f32", True, False, False),
    (20, 1, 264, "f32", False, False, False),
    (129, 3, 1000, "f32", True, False, False),
    (300, 4, 7168, "bf16", True, True, False),
    (17, 6, 264, "bf16", False, True, True),
    (41, 1, 1032, "bf16", False, True, False),
    (150, 2, 776, "bf16", True, False, False),   # 776 = 24 * 32 + 8: a block ends inside a slice's warp
    (97, 3, 1544, "bf16", True, True, True),
    (61, 5, 2056, "bf16", True, True, False),
    (23, 7, 520, "bf16", True, True, False),
    (9, 4, 8, "bf16", False, True, False),       # a row of one slice
    (9, 4, 4, "f32", False, True, False),
    (1000, 4, 1024, "bf16", True, True, False),  # several tokens and parameter batches a CTA
    (700, 2, 4096, "bf16", False, False, True),
    (6, 4, 16384, "bf16", True, True, False),
    (3, 2, 32768, "bf16", False, True, False),   # h not parked
    (3, 2, 16384, "f32", False, True, False),
])
def test_backward_matches_autograd(hc, T, n, d, dt, mix, read, shared):
    case = _backward_case(hc, T, n, d, dt, mix, read, shared, seed=100 + T + n)
    got = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    _check_backward(hc, got, *case)


@pytest.mark.parametrize("n,d,dt", [(4, 1024, "bf16"), (3, 1000, "f32"), (8, 512, "bf16"), (4, 7168, "bf16")])
def test_backward_without_dHout_or_gain(hc, n, d, dt):
    case = _backward_case(hc, 50, n, d, dt, True, True, False, 300, with_dHout=False, K=3)
    _check_backward(hc, hc.write_then_read_backward_checkpoint(*case[:8], **case[8]), *case)
    case = _backward_case(hc, 50, n, d, dt, False, True, False, 310, gain=False)
    got = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    assert got["dg"] is None
    _check_backward(hc, got, *case)
    case = _backward_case(hc, 50, n, d, dt, False, True, False, 320)
    got = hc.write_then_read_backward_checkpoint(*case[:8], want_dg=False, **case[8])
    assert got["dg"] is None
    _check_backward(hc, got, *case, sums=False)


# rows that are copied whole into shared memory: one to three slices a thread,
# two to four stages, rows at both ends of that range, fewer tokens than CTAs,
# several a CTA, and more than the parameter slots hold
@pytest.mark.parametrize("T,n,d,dt,mix,read,shared", [
    (1, 4, 7168, "bf16", True, True, False),
    (450, 4, 7168, "bf16", True, True, False),
    (149, 4, 5136, "bf16", False, True, True),
    (300, 3, 7664, "bf16", True, False, False),
    (300, 2, 7680, "bf16", True, True, False),
    (150, 1, 5136, "bf16", False, False, False),
    (300, 4, 2576, "f32", True, True, False),
    (150, 3, 3840, "f32", True, True, True),
    (2600, 3, 2592, "f32", False, True, False),
    (400, 2, 2592, "f32", True, False, False),
])
def test_backward_of_rows_in_shared_memory(hc, T, n, d, dt, mix, read, shared):
    case = _backward_case(hc, T, n, d, dt, mix, read, shared, seed=700 + T + n)
    got = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    again = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    for k in got:
        assert torch.equal(got[k], again[k]), k
    _check_backward(hc, got, *case)
    assert hc.device_fault() == 0


@pytest.mark.parametrize("n,d,dt", [(4, 5648, "bf16"), (2, 7168, "bf16"), (3, 2992, "f32")])
def test_backward_of_rows_in_shared_memory_without_dHout_or_gain(hc, n, d, dt):
    case = _backward_case(hc, 200, n, d, dt, True, True, False, 800, with_dHout=False, K=3)
    _check_backward(hc, hc.write_then_read_backward_checkpoint(*case[:8], **case[8]), *case)
    case = _backward_case(hc, 200, n, d, dt, False, True, False, 810, gain=False)
    _check_backward(hc, hc.write_then_read_backward_checkpoint(*case[:8], **case[8]), *case)


def test_backward_of_rows_in_shared_memory_on_streams_and_in_a_graph(hc):
    case = _backward_case(hc, 320, 4, 7168, "bf16", True, True, False, 820)
    other = _backward_case(hc, 310, 3, 5648, "bf16", False, True, False, 830)
    want = [hc.write_then_read_backward_checkpoint(*c[:8], **c[8]) for c in (case, other)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for c, s in zip((case, other), streams):
        with torch.cuda.stream(s):
            got.append(hc.write_then_read_backward_checkpoint(*c[:8], **c[8]))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for k in want[0]:
        assert torch.equal(got[0][k], want[0][k]) and torch.equal(got[1][k], want[1][k]), k
        assert torch.equal(out[k], want[0][k]), k


def test_backward_against_differences(hc):
    """Central differences of the fp64 step at the kept values, along random
    directions of every input (h^2 / 6 times the third derivative is below
    1e-6 at h = 1e-4). Bar: the roundings of the gradients' terms, four times
    their sum's size for the terms that cancel inside them."""
    T, n, d = 6, 3, 96
    case = _backward_case(hc, T, n, d, "f32", True, True, False, 400, K=4)
    cH, cy, A, b, a, g, dHo, dx, kw = case
    got = hc.write_then_read_backward_checkpoint(*case[:8], **kw)
    v = dict(dH=hc.checkpoint_unpack(cH, torch.float32), dy=hc.checkpoint_unpack(cy, torch.float32), dA=A, db=b, da=a,
             dg=g)
    v = {k: t.double().cpu() for k, t in v.items()}

    def loss(w):
        Hn, x = R.step(w["dH"], w["dy"], w["dA"], w["db"], w["da"], w["dg"], EPS, 1, kw["K"], 1)
        return float((Hn * dHo.double().cpu()).sum() + (x * dx.double().cpu()).sum())

    for i, k in enumerate(v):
        e = _normal(500 + i, *v[k].shape).double()
        h = 1e-4
        up, dn = dict(v), dict(v)
        up[k], dn[k] = v[k] + h * e, v[k] - h * e
        want = (loss(up) - loss(dn)) / (2 * h)
        terms = got[k].double().cpu() * e
        bar = 64 * R.U * float(terms.abs().sum()) * (1 + 2 * kw["K"] * (n + 1) / 64) * 4
        if k in ("dA", "da"):  # logits: the bar of each element, summed
            bar += 2e-4 * float(got[k].abs().max() * e.abs().sum())
        assert abs(float(terms.sum()) - want) <= bar + 1e-6, (k, float(terms.sum()), want)


def test_backward_shared_parameters_sum_over_tokens(hc):
    """Shared parameters give the per-token gradients of the same values given
    per token."""
    T, n, d = 90, 4, 1032
    cH, cy, A, b, a, g, dHo, dx, kw = _backward_case(hc, T, n, d, "bf16", True, True, True, 610)
    one = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    per = hc.write_then_read_backward_checkpoint(cH, cy, A.expand(T, n, n).contiguous(), b.expand(T, n).contiguous(),
                                                 a.expand(T, n).contiguous(), g, dHo, dx, **kw)
    for k in one:
        assert torch.equal(one[k], per[k]), k


def test_backward_strided_logits_of_one_projection(hc):
    """Parameters as slices of one [T, n*n + 2n] projection output."""
    T, n, d = 66, 4, 1024
    cH, cy, A, b, a, g, dHo, dx, kw = _backward_case(hc, T, n, d, "bf16", True, True, False, 620)
    P = torch.cat([A.reshape(T, n * n), a, b], 1).contiguous()
    got = hc.write_then_read_backward_checkpoint(cH, cy, P[:, :n * n].unflatten(1, (n, n)), P[:, n * n + n:],
                                                 P[:, n * n:n * n + n], g, dHo, dx, **kw)
    want = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    for k in want:
        assert torch.equal(got[k], want[k]), k


def test_backward_repeats_itself_on_another_stream_and_in_a_graph(hc):
    """The same bits on a side stream, in a captured graph replayed on new
    inputs, and for two calls at once with workspaces of their own."""
    T, n, d = 200, 4, 2048
    case = _backward_case(hc, T, n, d, "bf16", True, True, False, 630)
    other = _backward_case(hc, T, n, d, "bf16", True, True, False, 640)
    want = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    want2 = hc.write_then_read_backward_checkpoint(*other[:8], **other[8])
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s1):
        g1 = hc.write_then_read_backward_checkpoint(*case[:8], **case[8])
    with torch.cuda.stream(s2):
        g2 = hc.write_then_read_backward_checkpoint(*other[:8], **other[8])
    torch.cuda.synchronize()
    for k in want:
        assert torch.equal(g1[k], want[k]) and torch.equal(g2[k], want2[k]), k
    static = [None if t is None else (hc.Checkpoint(*(u.clone() for u in t)) if isinstance(t, tuple) else t.clone())
              for t in case[:8]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hc.write_then_read_backward_checkpoint(*static, **case[8])
    for src, ref in ((other, want2), (case, want)):
        for dst, t in zip(static, src[:8]):
            for x, z in zip(dst, t) if isinstance(t, tuple) else [(dst, t)]:
                x.view(torch.uint8).copy_(z.view(torch.uint8))
        graph.replay()
        torch.cuda.synchronize()
        for k in ref:
            assert torch.equal(out[k], ref[k]), k


def test_backward_not_finite_stays_in_its_token(hc):
    T, n, d = 300, 4, 1024
    cH, cy, A, b, a, g, dHo, dx, kw = _backward_case(hc, T, n, d, "bf16", True, True, False, 650)
    want = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    cH.codes.view(torch.uint8)[5, 2, 17] = 0x7F  # NaN
    dx2 = dx.clone()
    dx2[9, 3] = float("inf")
    got = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx2, **kw)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[5] = keep[9] = False
    for k in ("dH", "dy", "dA", "db", "da"):
        assert torch.equal(got[k][keep], want[k][keep]), k
        assert not got[k][5].isfinite().all(), k


def test_backward_past_32_bit_offsets(hc):
    """More than 2^31 stream values: the last tokens against autograd."""
    T, n, d = 75100, 4, 7168
    dev, gen = "cuda", torch.Generator(device="cuda").manual_seed(9)
    normal = lambda *s: torch.empty(s, dtype=torch.bfloat16, device=dev).normal_(generator=gen)
    cH, cy = hc.checkpoint_pack(normal(T, n, d)), hc.checkpoint_pack(normal(T, d))
    A, b, a = _params(71, T, n, False, True, True)
    g = torch.ones(d, device=dev)
    dHo, dx = normal(T, n, d), normal(T, d)
    kw = dict(eps=EPS, mix=0, K=0, read=1)
    got = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
    sl = slice(T - 3, T)
    cut = lambda c: hc.Checkpoint(c.codes[sl].contiguous(), c.scales[sl].contiguous())
    part = {k: (v[sl] if k != "dg" else v) for k, v in got.items()}
    _check_backward(hc, part, cut(cH), cut(cy), A, b, a, g, dHo[sl], dx[sl], kw, sums=False)


def test_training_steps_together(hc):
    """Three layers in place, forward with checkpoints and backward from them,
    against fp64 gradients of each layer at the values the checkpoints keep,
    chained. Three layers of 2 K (n + 1) + 64 roundings, on absolute sums of
    up to 8 times the row's rms (normal values: maxima of 4.5, doubled by the
    mix's non-negative weights)."""
    T, n, d, L, K = 70, 4, 1024, 3, 20
    x0 = _normal(80, T, d).cuda()
    H = hc.expand(x0, n)
    lay, saved = [], []
    for l in range(L):
        A, b, a = _params(90 + 5 * l, T, n, True, True, False)
        lay.append((A, b, a, (_normal(95 + l, d, std=0.2) + 1).cuda()))
        y = _normal(99 + l, T, d).cuda()
        H, x, cH, cy = hc.write_then_read_checkpoint(H, y, A, b, a, lay[l][3], mix=1, K=K, read=1, out=H)
        saved.append((cH, cy, x))
    dH = _normal(120, T, n, d).cuda()
    dxs = [_normal(121 + l, T, d).cuda() for l in range(L)]
    ref = dH.double()
    for l in reversed(range(L)):
        A, b, a, g = lay[l]
        got = hc.write_then_read_backward_checkpoint(saved[l][0], saved[l][1], A, b, a, g, dH, dxs[l], mix=1, K=K, read=1)
        kept = [hc.checkpoint_unpack(c, torch.float32).double() for c in saved[l][:2]]
        want = R.step_grads(*kept, A.double(), b.double(), a.double(), g.double(), EPS, ref, dxs[l], 1, K, 1)
        dH, ref = got["dH"], want["dH"]
        rms = ref.square().mean(-1, keepdim=True).sqrt()
        assert float(((dH.double() - ref).abs() / rms).max()) <= 3 * (2 * K * (n + 1) + 64) * R.U * 8


def test_refusals_on_the_gpu(hc):
    T, n, d = 8, 4, 64
    x = torch.zeros(T, n, d, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(T, d, device="cuda", dtype=torch.bfloat16)
    c, cy = hc.checkpoint_pack(x), hc.checkpoint_pack(y)
    A, b, a, g = torch.zeros(n, n, device="cuda"), *(torch.ones(k, device="cuda") for k in (n, n, d))
    bad = [
        (lambda: hc.checkpoint_pack(x.half()), ValueError),
        (lambda: hc.checkpoint_pack(x.transpose(0, 1)), ValueError),
        (lambda: hc.checkpoint_unpack(c, torch.float16), ValueError),
        (lambda: hc.checkpoint_unpack((c.codes, c.scales)), TypeError),
        (lambda: hc.checkpoint_unpack(hc.Checkpoint(c.codes, c.scales[..., :2])), ValueError),
        (lambda: hc.checkpoint_pack(x, out=cy), ValueError),
        (lambda: hc.write_then_read_checkpoint(x, y, A, b, a, H_ckpt=cy), ValueError),
        (lambda: hc.write_then_read_checkpoint(x, y.float(), A, b, a), ValueError),
        (lambda: hc.write_then_read_backward_checkpoint(c, c, A, b, a, g, None, y), ValueError),
        (lambda: hc.write_then_read_backward_checkpoint(c, cy, A, b, a, g, x.float(), y), ValueError),
        (lambda: hc.write_then_read_backward_checkpoint(c, cy, A, b, a, g.cpu(), None, y), ValueError),
    ]
    for call, err in bad:
        with pytest.raises(err):
            call()
    codes = [
        (lambda: hc.checkpoint_pack(torch.zeros(3, 12, device="cuda", dtype=torch.bfloat16)), hc.HC_ERR_UNSUPPORTED),
        (lambda: hc.checkpoint_pack(torch.zeros(65, device="cuda")[1:].view(2, 32)), hc.HC_ERR_MISALIGNED),
        (lambda: hc.write_then_read_checkpoint(x, y, A, b, a, out=x.view(-1)[:0].new_zeros(T, n, d), H_ckpt=c, y_ckpt=hc.Checkpoint(
            c.codes.view(-1)[:T * d].view(T, d), cy.scales)), hc.HC_ERR_ALIAS),
        (lambda: hc.write_then_read_backward_checkpoint(c, cy, A, b, a, g, None, y, workspace=torch.empty(
            16, dtype=torch.uint8, device="cuda")), hc.HC_ERR_INVALID_ARG),
        (lambda: hc.write_then_read_backward_checkpoint(c, cy, A, b, a, g, None, y, mix=1, K=5000), hc.HC_ERR_UNSUPPORTED),
    ]
    for call, status in codes:
        with pytest.raises(hc.HCError) as e:
            call()
        assert e.value.status == status
    out = hc.write_then_read_backward_checkpoint(hc.checkpoint_pack(x[:0]), hc.checkpoint_pack(y[:0]), A, b, a, g, None, y[:0])
    assert out["dH"].shape == (0, n, d) and (out["dg"] == 0).all()
    H0, x0, c0, _ = hc.write_then_read_checkpoint(x[:0], y[:0], A, b, a)
    assert H0.shape == (0, n, d) and c0.codes.shape == (0, n, d)
