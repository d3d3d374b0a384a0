"""Refusals of the training entry points, without a GPU: statuses for bad
arguments (fake device addresses, in a child process that sees no device), and
the binding's refusal of host tensors."""
from __future__ import annotations

import json
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = textwrap.dedent(r"""
    import json
    from hyper_connections_stream_b200 import _lib as B
    L = B.lib()
    def buf(i): return 0x10000 * (i + 1) * 4096     # fake, aligned, never dereferenced
    res = {}
    def call(tag, fn, *args):
        res[tag] = (getattr(L, fn)(*args), L.hc_last_error().decode())
    T, n, d = 8, 4, 1024
    H, y, Ho, x, A, b, a, g, q, s, qy, sy, dH, dy, dA, db, da, dg, ws, dx, dHo, beta = (buf(i) for i in range(22))
    bf, f32, inf, nan = B.HC_BF16, B.HC_F32, float("inf"), float("nan")
    big = 1 << 40

    def pack(tag, X=H, dt=bf, rows=T * n, dd=d, qq=q, ss=s):
        call("pk_" + tag, "hc_checkpoint_pack", X, dt, rows, dd, qq, ss, None)
        call("up_" + tag, "hc_checkpoint_unpack", qq, ss, X, dt, rows, dd, None)
    pack("dtype", dt=7)
    pack("rows_neg", rows=-1)
    pack("rows_0", X=None, qq=None, ss=None, rows=0)
    pack("d_0", dd=0)
    pack("d_ragged", dd=12)
    pack("d_big", dd=(1 << 30) + 8, rows=1)
    pack("too_many", rows=1 << 62)
    pack("null_X", X=None)
    pack("null_q", qq=None)
    pack("null_s", ss=None)
    pack("mis_X", X=H + 8)
    pack("mis_q", qq=q + 8)
    pack("mis_s", ss=s + 4)
    pack("alias_q", qq=H + 16)
    call("pk_alias_qs", "hc_checkpoint_pack", H, bf, T * n, d, q, q + T * n * d - 16, None)

    def step(tag, Hh=H, yy=y, out=Ho, xx=x, dt=bf, t=T, nn=n, dd=d, mm=0, Aa=A, As=0, K=0, bb=b, rm=0, aa=a, gg=None,
             eps=1e-6, q1=q, s1=s, q2=qy, s2=sy):
        call("st_" + tag, "hc_write_then_read_checkpoint", Hh, yy, out, xx, dt, t, nn, dd, mm, Aa, As, K, bb, 0, rm,
             aa, 0, gg, eps, q1, s1, q2, s2, None)
    step("T0", Hh=None, yy=None, out=None, xx=None, t=0, q1=None, s1=None, q2=None, s2=None)
    step("n9", nn=9)
    step("d_ragged", dd=12)
    step("d_big", dd=32776)
    step("mix", mm=3)
    step("read", rm=2)
    step("K0", mm=1)
    step("stride", As=-1)
    step("eps", eps=nan)
    step("null_q", q1=None)
    step("null_sy", s2=None)
    step("mis_q", q1=q + 8)
    step("mis_sy", s2=sy + 8)
    step("mis_g", gg=g + 4)
    step("alias_q_H", q1=H + 16)
    step("alias_q_Hout", q1=Ho + 16)
    step("alias_qy_x", q2=x)
    step("alias_q_qy", q2=q + 64)
    step("alias_part", out=H + 16)
    step("alias_A", s1=A)

    def back(tag, q1=q, s1=s, q2=qy, s2=sy, dt=bf, t=T, nn=n, dd=d, mm=0, Aa=A, K=0, bb=b, rm=0, aa=a, gg=g, eps=1e-6,
             do=dHo, di=dx, o1=dH, o2=dy, o3=dA, o4=db, o5=da, o6=dg, w=ws, wb=big):
        call("bw_" + tag, "hc_write_then_read_backward_checkpoint", q1, s1, q2, s2, dt, t, nn, dd, mm, Aa, 0, K, bb, 0,
             rm, aa, 0, gg, eps, do, di, o1, o2, o3, o4, o5, o6, w, wb, None)
    back("T0", q1=None, s1=None, q2=None, s2=None, t=0, do=None, di=None, o1=None, o2=None, o6=None)
    back("n0", nn=0)
    back("d_ragged_f32", dt=f32, dd=6)
    back("mix", mm=-1)
    back("read", rm=9)
    back("K0", mm=1)
    back("eps", eps=inf)
    back("null_q", q1=None)
    back("null_s", s1=None)
    back("null_qy", q2=None)
    back("null_dx", di=None)
    back("null_dH", o1=None)
    back("null_dA", o3=None)
    back("mis_dHout", do=dHo + 8)
    back("mis_s", s1=s + 8)
    back("dg_no_g", gg=None)
    back("dg_no_ws", w=None)
    back("mis_ws", w=ws + 8, wb=1 << 20)
    back("alias_dH_q", o1=q, wb=0)
    back("alias_dH_dHout", o1=dHo, wb=0)
    back("alias_dH_dy", o2=dH + 64, wb=0)
    back("alias_dA_A", o3=A, wb=0)

    def ln(tag, Hh=H, xx=x, dt=bf, t=T, nn=n, dd=d, rm=0, aa=a, st=0, gg=None, bb=None, eps=1e-6):
        call("ln_" + tag, "hc_read_layernorm", Hh, xx, dt, t, nn, dd, rm, aa, st, gg, bb, eps, None)
    ln("T0", Hh=None, xx=None, t=0)
    ln("dtype", dt=2)
    ln("d_big", dd=32776)
    ln("read", rm=4)
    ln("stride", st=-4)
    ln("eps", eps=-1.0)
    ln("null_H", Hh=None)
    ln("null_a", aa=None)
    ln("mis_x", xx=x + 2)
    ln("mis_g", gg=g + 8)
    ln("mis_beta", bb=beta + 8)
    ln("alias", xx=H + 32)
    ln("alias_beta", bb=x)

    def lb(tag, Hh=H, ss=None, dt=bf, t=T, nn=n, dd=d, rm=0, aa=a, gg=g, eps=1e-6, di=dx, o1=dH, o2=da, o3=dg,
           o4=beta, w=ws, wb=big):
        call("lb_" + tag, "hc_read_layernorm_backward", Hh, ss, dt, t, nn, dd, rm, aa, 0, gg, eps, di, o1, o2, o3, o4,
             w, wb, None)
    lb("T0", Hh=None, t=0, di=None, o1=None, o3=None, o4=None)
    lb("n9", nn=9)
    lb("read", rm=4)
    lb("eps", eps=nan)
    lb("null_H", Hh=None)
    lb("null_dx", di=None)
    lb("mis_s", ss=s + 8)
    lb("null_a", aa=None, o2=None)
    lb("da_no_a", aa=None, nn=1)
    lb("mis_da", o2=da + 2)
    lb("dg_no_g", gg=None)
    lb("no_ws", w=None)
    lb("mis_dbeta", o4=beta + 2)
    lb("alias_dH_H", o1=H, wb=0)
    lb("alias_dH_codes", ss=s, o1=H + 16, wb=0)
    lb("alias_dg_dbeta", o3=dg, o4=dg + 16, wb=0)
    lb("alias_ws_dH", w=dH + 16, wb=64)
    print(json.dumps(res))
""")


def test_argument_validation_statuses():
    from hyper_connections_stream_b200 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, "-c", _CHILD], capture_output=True, text=True, env=env, cwd=ROOT, timeout=300)
    assert out.returncode == 0, out.stderr
    res = json.loads(out.stdout.strip().splitlines()[-1])
    OK, INV, UNS, MIS, ALI = 0, 1, 2, 3, 4
    for tag, (got, msg) in res.items():
        kind = tag.split("_", 1)[1]
        if kind in ("rows_0", "T0"):
            code = OK
        elif kind.startswith("mis_"):
            code = MIS
        elif kind.startswith("alias"):
            code = ALI
        elif kind in ("n9", "d_ragged", "d_ragged_f32", "d_big"):
            code = UNS
        else:
            code = INV
        assert got == code, (tag, got, code, msg)
        assert (got == OK) or msg, tag
    assert len(res) > 90


def test_scale_stride():
    from hyper_connections_stream_b200 import _lib
    L = _lib.lib()
    for d, want in ((0, 0), (-3, 0), (4, 16), (32, 16), (512, 16), (516, 32), (7168, 224), (7200, 240), (32768, 1024)):
        assert L.hc_checkpoint_scale_stride(d) == want == _lib.checkpoint_scale_stride(d), d


def test_binding_refuses_host_tensors_and_foreign_types():
    from hyper_connections_stream_b200 import _lib as hc
    H = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    y = torch.zeros((2, 64), dtype=torch.bfloat16)
    c, cy = hc.checkpoint_empty((2, 4, 64), "cpu"), hc.checkpoint_empty((2, 64), "cpu")
    A, a, g = torch.eye(4), torch.ones(4), torch.ones(64)
    for call in (lambda: hc.checkpoint_pack(H), lambda: hc.checkpoint_unpack(c),
                 lambda: hc.write_then_read_checkpoint(H, y, A, a, a),
                 lambda: hc.write_then_read_backward_checkpoint(c, cy, A, a, a, g, None, y),
                 lambda: hc.read_layernorm(H, a, g), lambda: hc.read_layernorm_backward(H, a, g, y),
                 lambda: hc.read_layernorm_backward(c, a, g, y)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        hc.checkpoint_unpack(H)
    assert c.scales.shape == (2, 4, 16) and c.codes.dtype == torch.float8_e4m3fn


def test_reference_codes():
    """The tests' own e4m3 table and search against torch's conversion."""
    from tests import _train_ref as R
    v = R.e4m3_values()
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    x = np.random.default_rng(3).standard_normal((4, 96)) * 10.0 ** np.arange(-2, 2)[:, None]
    kept, e = R.pack_ref(x)
    s = np.repeat(2.0 ** (e.astype(float) - 127), 32, axis=-1)
    want = torch.from_numpy(x / s).float().to(torch.float8_e4m3fn).double().numpy() * s
    assert np.abs(kept - want).max() <= 2.0 ** -20 * np.abs(x).max()
    assert np.abs(x / s).max() <= 448 and (np.abs(x / s).reshape(4, 3, 32).max(-1) > 224).all()
