"""fp64 definitions of the training operators for their tests (torch, any
device, no library code): 8-bit checkpoints, the step and its gradients, the
layer-norm read and its gradients. Gradients come from autograd of the
forwards below; error bounds come from the same formulas with absolute values.

U is fp32's unit roundoff 2^-24. A bound C * U * (sum of the absolute values
that enter a result) allows C roundings on every one of them.
"""
from __future__ import annotations

import numpy as np
import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}  # storage rounding, relative


# ---- 8-bit checkpoints --------------------------------------------------------

def e4m3_values() -> np.ndarray:
    """The value of every e4m3 code 0..255 (codes 127 and 255 are NaN)."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def pack_ref(x: np.ndarray):
    """Kept values (fp64) and biased scale exponents [.., blocks] of x [.., d]
    (fp64 values of the stored tensor), by search over the 127 finite
    magnitudes: nearest, ties to the even code."""
    d = x.shape[-1]
    nb = -(-d // 32)
    b = np.zeros((*x.shape[:-1], nb * 32))
    b[..., :d] = x
    b = b.reshape(*x.shape[:-1], nb, 32)
    fin = np.isfinite(b)
    amax = np.max(np.where(fin, np.abs(b), 0.0), axis=-1)
    e = np.full(amax.shape, -126)
    while True:
        up = amax / 2.0 ** e > 448.0
        if not up.any():
            break
        e = e + up
    s = 2.0 ** e[..., None].astype(np.float64)
    mags = e4m3_values()[:127]
    a = np.abs(np.where(fin, b, 0.0)) / s
    hi = np.clip(np.searchsorted(mags, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mags[lo], mags[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    kept = np.copysign(mags[pick], b) * s
    kept = np.where(fin, kept, np.nan)
    return kept.reshape(*x.shape[:-1], nb * 32)[..., :d], (e + 127).astype(np.uint8)


# ---- the step -------------------------------------------------------------------

def project(L, K):
    M = torch.exp(L)
    for _ in range(K):
        M = M / M.sum(-1, keepdim=True)
        M = M / M.sum(-2, keepdim=True)
    return M


def step(H, y, A, b, a, g, eps, mix, K, read):
    """(H', x) of the step, nothing rounded. Leading token axis on H, y; the
    parameters per token or shared."""
    T, n, _ = H.shape
    Am = project(A, K) if mix else A
    aw = torch.softmax(a, -1) if read else a
    Am, aw, bw = Am.expand(T, n, n), aw.expand(T, n), b.expand(T, n)
    Hn = torch.einsum("tij,tid->tjd", Am, H) + bw[:, :, None] * y[:, None]
    h = torch.einsum("tj,tjd->td", aw, Hn)
    x = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    return Hn, x if g is None else x * g


def per_token(p, T, dims):
    """A per-token fp64 copy of a parameter (gradients come per token)."""
    p = p.double()
    return p.expand(T, *p.shape).clone() if p.dim() == dims else p.clone()


def step_grads(H, y, A, b, a, g, eps, dHout, dx, mix, K, read):
    """Gradients of <dHout, H'> + <dx, x> (autograd, fp64)."""
    T = H.shape[0]
    v = dict(dH=H.double().clone(), dy=y.double().clone(), dA=per_token(A, T, 2), db=per_token(b, T, 1),
             da=per_token(a, T, 1))
    if g is not None:
        v["dg"] = g.double().clone()
    for t in v.values():
        t.requires_grad_(True)
    Hn, x = step(v["dH"], v["dy"], v["dA"], v["db"], v["da"], v.get("dg"), eps, mix, K, read)
    loss = (x * dx.double()).sum()
    if dHout is not None:
        loss = loss + (Hn * dHout.double()).sum()
    grads = torch.autograd.grad(loss, list(v.values()))
    return dict(zip(v, grads))


def step_bounds(H, y, A, b, a, g, eps, dHout, dx, mix, K, read):
    """The same gradients with every product taken by its absolute value."""
    T, n, d = H.shape
    H, y, dx = H.double(), y.double(), dx.double()
    Am = (project(A.double(), K) if mix else A.double()).expand(T, n, n)
    aw = (torch.softmax(a.double(), -1) if read else a.double()).expand(T, n)
    bw = b.double().expand(T, n)
    c = torch.einsum("tij,tj->ti", Am, aw)
    cy = (bw * aw).sum(-1)
    h = torch.einsum("ti,tid->td", c, H) + cy[:, None] * y
    ha = torch.einsum("tij,tj,tid->td", Am.abs(), aw.abs(), H.abs()) + ((bw * aw).abs().sum(-1))[:, None] * y.abs()
    r = 1.0 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    u = dx.abs() * (1.0 if g is None else g.double().abs())
    dh = r * u + r ** 3 * (u * ha).mean(-1, keepdim=True) * ha
    G = (0.0 if dHout is None else dHout.double().abs()) + aw.abs()[:, :, None] * dh[:, None]
    P = torch.einsum("td,tid->ti", dh, H.abs())
    Py = (dh * y.abs()).sum(-1)
    return dict(dH=torch.einsum("tij,tjd->tid", Am.abs(), G), dy=torch.einsum("tj,tjd->td", bw.abs(), G),
                dA=torch.einsum("tid,tjd->tij", H.abs(), G), db=torch.einsum("td,tjd->tj", y.abs(), G),
                da=torch.einsum("tij,ti->tj", Am.abs(), P) + bw.abs() * Py[:, None],
                dg=(dx.abs() * ha * r).sum(0))


# ---- the layer-norm read ----------------------------------------------------------

def layernorm(H, a, g, beta, eps, read):
    T, n, _ = H.shape
    aw = torch.ones(n, dtype=H.dtype, device=H.device) if a is None else torch.softmax(a, -1) if read else a
    h = torch.einsum("tn,tnd->td", aw.expand(T, n), H)
    h = h - h.mean(-1, keepdim=True)
    x = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    x = x if g is None else x * g
    return x if beta is None else x + beta


def layernorm_grads(H, a, g, eps, dx, read):
    T, n, d = H.shape
    v = dict(dH=H.double().clone(), dbeta=torch.zeros(d, dtype=torch.float64, device=H.device))
    if a is not None:
        v["da"] = per_token(a, T, 1)
    if g is not None:
        v["dg"] = g.double().clone()
    for t in v.values():
        t.requires_grad_(True)
    x = layernorm(v["dH"], v.get("da"), v.get("dg"), v["dbeta"], eps, read)
    return dict(zip(v, torch.autograd.grad((x * dx.double()).sum(), list(v.values()))))


def layernorm_bounds(H, a, g, beta, eps, dx, read):
    """Absolute-value sums for x and the gradients. s * (sum |a_i H_i| +
    |mean|) is what a rounding of h or of the mean does to the normalised
    value."""
    T, n, d = H.shape
    H = H.double()
    aw = torch.ones(n, dtype=H.dtype, device=H.device) if a is None else \
        torch.softmax(a.double(), -1) if read else a.double()
    aw = aw.expand(T, n)
    h = torch.einsum("tn,tnd->td", aw, H)
    mu = h.mean(-1, keepdim=True)
    s = 1.0 / torch.sqrt(((h - mu) ** 2).mean(-1, keepdim=True) + eps)
    ha = torch.einsum("tn,tnd->td", aw.abs(), H.abs())
    z = s * (ha + mu.abs())
    ga = 1.0 if g is None else g.double().abs()
    out = dict(x=z * ga + (0.0 if beta is None else beta.double().abs()))
    if dx is not None:
        u = dx.double().abs() * ga
        dh = s * (u + u.mean(-1, keepdim=True) + z * (u * z).mean(-1, keepdim=True))
        out.update(dH=aw.abs()[:, :, None] * dh[:, None], da=torch.einsum("td,tnd->tn", dh, H.abs()),
                   dg=(dx.double().abs() * z).sum(0), dbeta=dx.double().abs().sum(0))
        if read:
            out["da"] = out["da"] + out["da"].sum(-1, keepdim=True)
    return out


def check_as(what, got, ref, bound, roundings, step):
    """|got - ref| <= roundings * U * bound + step * |ref|; NaN exactly where
    ref has it."""
    got, ref, bound = got.detach().double().cpu(), ref.detach().double().cpu(), bound.double().cpu()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(got.isnan(), ref.isnan()), f"{what}: NaN in other places"
    off = (got - ref).abs()
    lim = roundings * U * bound + step * ref.abs() * (1 + 2.0 ** -6) + 1e-37
    bad = off > lim
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / lim).nan_to_num().max()):.2f}"
                           f" times the bound")
