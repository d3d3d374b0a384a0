"""Calls of the training entry points that a program makes around the ordinary
ones: outputs inside larger buffers that hold something already, a workspace of
exactly the queried size full of NaN, strided read weights, and a first call
that is captured into a graph. Bits are compared with those of the plain calls."""
from __future__ import annotations

import os
import subprocess
import sys
import textwrap

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
PAD = 4096  # bytes kept on either side of an output


@pytest.fixture(scope="module")
def hc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from hyper_connections_stream_b200 import build
    build.build()
    import hyper_connections_stream_b200._lib as L
    L.lib()
    L.set_path(L.PATH_AUTO)
    yield L
    L.set_path(L.PATH_AUTO)
    torch.cuda.synchronize()
    assert L.device_fault() == 0


def _normal(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


class _Guarded:
    """Buffers inside larger ones: NaN bytes (0xFF) inside, 0xA5 around."""

    def __init__(self):
        self.bufs = []

    def make(self, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        n = t.numel() * t.element_size()
        raw = torch.full((n + 2 * PAD + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        raw[PAD:PAD + n] = 0xFF
        self.bufs.append((raw, n))
        return raw[PAD:PAD + n].view(dtype).view(shape)

    def intact(self):
        return all(bool((r[:PAD] == 0xA5).all()) and bool((r[PAD + n:] == 0xA5).all()) for r, n in self.bufs)


def _bits(t):
    return t.contiguous().view(torch.uint8)


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _ok(hc, status):
    assert status == hc.HC_OK, hc.lib().hc_last_error()


@pytest.mark.parametrize("T,n,d,dt", [(37, 4, 1024, "bf16"), (300, 4, 7168, "bf16"), (33, 8, 520, "bf16"),
                                      (155, 2, 2592, "f32"), (700, 3, 1000, "f32"), (3, 2, 32768, "bf16"),
                                      (400, 1, 1032, "bf16"), (1, 4, 5136, "bf16")])
def test_backward_from_a_checkpoint_between_neighbours(hc, T, n, d, dt):
    cH, cy = hc.checkpoint_pack(_normal(1, T, n, d)), hc.checkpoint_pack(_normal(2, T, d))
    A, b, a, g = _normal(3, T, n, n), _normal(4, n), _normal(5, T, n), _normal(6, d)
    dHo, dx = _normal(7, T, n, d).to(DT[dt]), _normal(8, T, d).to(DT[dt])
    want = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, mix=1, K=5, read=1)
    G = _Guarded()
    out = {k: G.make(v.shape, v.dtype) for k, v in want.items()}
    need = hc.lib().hc_write_then_read_backward_checkpoint_workspace_bytes(hc._DT[DT[dt]], T, n, d)
    ws = G.make((need,), torch.uint8)
    _ok(hc, hc.lib().hc_write_then_read_backward_checkpoint(
        cH.codes.data_ptr(), cH.scales.data_ptr(), cy.codes.data_ptr(), cy.scales.data_ptr(), hc._DT[DT[dt]], T, n, d, 1,
        A.data_ptr(), n * n, 5, b.data_ptr(), 0, 1, a.data_ptr(), n, g.data_ptr(), 1e-6, dHo.data_ptr(), dx.data_ptr(),
        *(out[k].data_ptr() for k in ("dH", "dy", "dA", "db", "da", "dg")), ws.data_ptr(), need, _stream()))
    for k in want:
        assert torch.equal(_bits(out[k]), _bits(want[k])), k
    assert G.intact()
    with pytest.raises(hc.HCError) as e:
        hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, mix=1, K=5, read=1, workspace=ws[:-16])
    assert e.value.status == hc.HC_ERR_INVALID_ARG


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("T,n,d,dt", [(37, 4, 1024, "bf16"), (300, 1, 7168, "bf16"), (160, 4, 7168, "bf16"),
                                      (33, 8, 520, "bf16"), (155, 2, 3584, "f32"), (700, 3, 1004, "f32"),
                                      (3, 2, 32768, "bf16"), (900, 2, 72, "bf16"), (1, 1, 8, "bf16")])
def test_layernorm_backward_between_neighbours(hc, T, n, d, dt, packed):
    H, a, g = _normal(11, T, n, d, mean=0.3).to(DT[dt]), _normal(12, T, n), _normal(13, d)
    dx = _normal(14, T, d).to(DT[dt])
    src = hc.checkpoint_pack(H) if packed else H
    want = hc.read_layernorm_backward(src, a, g, dx, read=1)
    G = _Guarded()
    out = {k: G.make(v.shape, v.dtype) for k, v in want.items()}
    need = hc.lib().hc_read_layernorm_backward_workspace_bytes(hc._DT[DT[dt]], T, n, d)
    ws = G.make((need,), torch.uint8)
    rows, scales = (src.codes, src.scales.data_ptr()) if packed else (src, None)
    _ok(hc, hc.lib().hc_read_layernorm_backward(
        rows.data_ptr(), scales, hc._DT[DT[dt]], T, n, d, 1, a.data_ptr(), n, g.data_ptr(), 1e-6, dx.data_ptr(),
        *(out[k].data_ptr() for k in ("dH", "da", "dg", "dbeta")), ws.data_ptr(), need, _stream()))
    for k in want:
        assert torch.equal(_bits(out[k]), _bits(want[k])), k
    assert G.intact()


@pytest.mark.parametrize("T,n,d,dt,path", [(300, 4, 4096, "bf16", "pipelined"), (300, 3, 1000, "f32", "pipelined"),
                                           (37, 8, 1032, "bf16", "pipelined"), (37, 8, 1032, "bf16", "register"),
                                           (300, 4, 1028, "f32", "register"), (1, 2, 8, "bf16", "pipelined"),
                                           (5, 1, 264, "bf16", "register")])
def test_saving_step_between_neighbours(hc, T, n, d, dt, path):
    H, y = _normal(21, T, n, d).to(DT[dt]), _normal(22, T, d).to(DT[dt])
    A, b, a, g = _normal(23, T, n, n), _normal(24, n), _normal(25, T, n), _normal(26, d)
    hc.set_path(hc.PATH_PIPELINED if path == "pipelined" else hc.PATH_REGISTER)
    want = hc.write_then_read_checkpoint(H, y, A, b, a, g, mix=1, K=5, read=1)
    G = _Guarded()
    ns = hc.checkpoint_scale_stride(d)
    out, x = G.make((T, n, d), DT[dt]), G.make((T, d), DT[dt])
    cH = hc.Checkpoint(G.make((T, n, d), torch.float8_e4m3fn), G.make((T, n, ns), torch.uint8))
    cy = hc.Checkpoint(G.make((T, d), torch.float8_e4m3fn), G.make((T, ns), torch.uint8))
    got = hc.write_then_read_checkpoint(H, y, A, b, a, g, mix=1, K=5, read=1, out=out, x_next=x, H_ckpt=cH, y_ckpt=cy)
    nb = -(-d // 32)
    for p, q in zip(got[:2], want[:2]):
        assert torch.equal(_bits(p), _bits(q))
    for p, q in zip(got[2:], want[2:]):
        assert torch.equal(_bits(p.codes), _bits(q.codes))
        assert torch.equal(p.scales[..., :nb], q.scales[..., :nb])
        assert (p.scales[..., nb:] == 0xFF).all()
    assert G.intact()


@pytest.mark.parametrize("T,n,d", [(300, 4, 1024), (200, 4, 7168)])
def test_layernorm_of_strided_weights(hc, T, n, d):
    """Read weights as a slice of one [T, n * n + 2 n] projection output."""
    P = _normal(31, T, n * n + 2 * n)
    a, H, dx = P[:, n * n:n * n + n], _normal(32, T, n, d).bfloat16(), _normal(33, T, d).bfloat16()
    g = _normal(34, d)
    assert torch.equal(hc.read_layernorm(H, a, g, read=1), hc.read_layernorm(H, a.contiguous(), g, read=1))
    for src in (H, hc.checkpoint_pack(H)):
        got = hc.read_layernorm_backward(src, a, g, dx, read=1)
        want = hc.read_layernorm_backward(src, a.contiguous(), g, dx, read=1)
        for k in want:
            assert torch.equal(got[k], want[k]), k


_CHILD = textwrap.dedent(r"""
    import torch
    from hyper_connections_stream_b200 import _lib as hc
    T, n, d = 200, 4, 5136
    gen = torch.Generator(device="cuda").manual_seed(1)
    N = lambda *s: torch.randn(*s, generator=gen, device="cuda")
    H, y, A, b, a, g = N(T, n, d).bfloat16(), N(T, d).bfloat16(), N(T, n, n), N(n), N(T, n), N(d)
    dHo, dx, kw = N(T, n, d).bfloat16(), N(T, d).bfloat16(), dict(mix=1, K=20, read=1)
    def step():
        Hn, x, cH, cy = hc.write_then_read_checkpoint(H, y, A, b, a, g, **kw)
        gr = hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, dHo, dx, **kw)
        z = hc.read_layernorm(Hn, a, g, read=1)
        lr = hc.read_layernorm_backward(cH, a, g, dx, read=1)
        kept = hc.checkpoint_unpack(cH)
        return [Hn, x, z, kept, *gr.values(), *lr.values()]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    graph.replay()
    torch.cuda.synchronize()
    want = step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))
    print("same")
""")


def test_first_calls_captured(hc):
    """In a fresh process every call's first time is inside a capture."""
    out = subprocess.run([sys.executable, "-c", _CHILD], capture_output=True, text=True, cwd=ROOT, timeout=300,
                         env=dict(os.environ, PYTHONPATH=ROOT))
    assert out.returncode == 0 and "same" in out.stdout, (out.stdout[-1000:], out.stderr[-3000:])
