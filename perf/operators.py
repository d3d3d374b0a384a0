"""Cases of the training operators: 8-bit stream checkpoints and the gradients taken from them, layer-norm reads and
their gradients.

`run` computes a case in its plain form (elementary torch operations in fp32, rounded once) or, with `own` set, through
the library's entry points. `exact` gives the same results from the definitions in fp64. Sizes follow the repository's
own configurations (d = 7168 and 4096, n = 1 .. 8 streams, up to 16384 tokens) and odd sizes between them.

Definitions, for one token (H [n][d] streams, y [d] block output, fp32 parameters):
  checkpoint   blocks of 32 along d; 2^e the smallest power of two with max|x| / 2^e <= 448 (e >= -126), value kept
               e4m3(x / 2^e) * 2^e
  step         H'_j = rnd(sum_i A_ij H_i + b_j y), x = h (mean h^2 + eps)^-1/2 g with h = sum_j a_j H'_j; its
               gradients are taken at the checkpoint's H and y, where H' is not rounded
  layer norm   x = (h - mean h)(var h + eps)^-1/2 g + beta with h = sum_i a_i H_i
  parameters   "logits": A = Sinkhorn(L) (K times divide rows, then columns, by their sums), a = softmax(l), per token;
               "matrix": A, a as given, one set for all tokens
"""
import math

import torch

own = False

EPS = 1e-6
K = 20
BLOCK = 32
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one ragged micro-batch put away and brought back: launch latency, blocks that end inside a row
        {"name": "pack_ragged", "op": "pack", "T": 37, "n": 4, "d": 1032, "dt": "bf16"},
        # the streams of one layer of the large model, a whole batch
        {"name": "pack_layer", "op": "pack", "T": 16384, "n": 4, "d": 7168, "dt": "bf16"},
        # a training step of a small fp32 model, odd token count
        {"name": "step_small_f32", "op": "step", "T": 129, "n": 3, "d": 1000, "dt": "f32", "mix": "logits"},
        # a training step of the static layer
        {"name": "step_static", "op": "step", "T": 4096, "n": 4, "d": 4096, "dt": "bf16", "mix": "matrix"},
        # a training step of the large model's layer, per-token mixing
        {"name": "step_mhc", "op": "step", "T": 8192, "n": 4, "d": 7168, "dt": "bf16", "mix": "logits"},
        # the backward alone, as the second half of a step runs it
        {"name": "backward_mhc", "op": "backward", "T": 16384, "n": 4, "d": 7168, "dt": "bf16", "mix": "logits"},
        # the widest state
        {"name": "backward_wide", "op": "backward", "T": 2048, "n": 8, "d": 4096, "dt": "bf16", "mix": "logits"},
        # one token of decoding
        {"name": "ln_decode", "op": "ln", "T": 1, "n": 4, "d": 7168, "dt": "bf16", "mix": "logits"},
        # a batch of prompts
        {"name": "ln_prompt", "op": "ln", "T": 16384, "n": 4, "d": 4096, "dt": "bf16", "mix": "logits"},
        # the plain layer norm's gradient (one stream, no read weights)
        {"name": "ln_backward_plain", "op": "ln_backward", "T": 16384, "n": 1, "d": 7168, "dt": "bf16",
         "mix": "none", "packed": False},
        # a layer's read from its checkpoint
        {"name": "ln_backward_packed", "op": "ln_backward", "T": 8192, "n": 4, "d": 7168, "dt": "bf16",
         "mix": "logits", "packed": True},
        # a small fp32 model, ragged
        {"name": "ln_backward_f32", "op": "ln_backward", "T": 257, "n": 2, "d": 1000, "dt": "f32",
         "mix": "matrix", "packed": False},
    ]


def draw(rng):
    op = rng.choice(["pack", "step", "backward", "ln", "ln_backward"])
    dt = rng.choice(["bf16", "bf16", "f32"])
    # at n = 1 a read weight has no gradient but rounding (the norm cancels it): those steps are left out
    n = rng.choice([2, 3, 4, 4, 6, 8] if op in ("step", "backward") else [1, 1, 2, 3, 4, 4, 6, 8])
    v = 8 if dt == "bf16" else 4
    d = max(v, int(math.exp(rng.uniform(math.log(256), math.log(7168)))) // v * v)
    if rng.random() < 0.4:
        d = rng.choice([1024, 2048, 4096, 7168])
    most = min(16384, 16384 * 4 * 7168 // (2 * n * d))
    T = int(math.exp(rng.uniform(0.0, math.log(most))))
    case = {"op": op, "T": T, "n": n, "d": d, "dt": dt}
    if op != "pack":
        case["mix"] = rng.choice(["logits", "matrix"])
    if op in ("ln", "ln_backward") and n == 1:
        case["mix"] = "none"
    if op == "ln_backward":
        case["packed"] = rng.random() < 0.5
    while work(case)["bytes"] > 2.9e9:
        case["T"] = case["T"] * 3 // 4
    return case


# ---- inputs -------------------------------------------------------------------

def _streams(gen, shape, dt, offset=0.0):
    """Values of a residual stream: normal, every channel with a size of its own, a few channels much larger."""
    x = torch.empty(shape, device="cuda")
    x.normal_(generator=gen)
    size = torch.empty(shape[-1], device="cuda").normal_(0.0, 0.5, generator=gen).exp_()
    big = torch.empty(shape[-1], device="cuda").uniform_(generator=gen) < 0.002
    x.mul_(torch.where(big, 20.0 * size, size)).add_(offset)
    return x.to(_DT[dt])


def _blocks(x):
    """fp32 [.., d] -> [.., blocks, 32], zeros behind the last value."""
    d = x.shape[-1]
    nb = -(-d // BLOCK)
    return torch.nn.functional.pad(x, (0, nb * BLOCK - d)).unflatten(-1, (nb, BLOCK))


def _pack(x):
    """e4m3 codes [.., d] and one biased exponent a block [.., nb padded to a multiple of 16]."""
    b = _blocks(x.float())
    amax = b.abs().amax(-1)
    bits = amax.view(torch.int32)
    e = (((bits + 0x1FFFFF) >> 23) - 8).clamp(min=1)
    inv = ((254 - e) << 23).view(torch.float32)
    q = (b * inv.unsqueeze(-1)).to(torch.float8_e4m3fn).flatten(-2)[..., : x.shape[-1]].contiguous()
    s = torch.nn.functional.pad(e.to(torch.uint8), (0, -e.shape[-1] % 16))
    return q, s.contiguous()


def _unpack(q, s):
    """fp32 values of a checkpoint."""
    d = q.shape[-1]
    scale = (s[..., : -(-d // BLOCK)].int() << 23).view(torch.float32)
    return (_blocks(q.float()) * scale.unsqueeze(-1)).flatten(-2)[..., :d]


def prepare(case, seed):
    T, n, d, dt, op = case["T"], case["n"], case["d"], case["dt"], case["op"]
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))

    def normal(*shape, mean=0.0, std=1.0):
        return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen)

    st = {"case": case, "H": _streams(gen, (T, n, d), dt, 0.25 if op.startswith("ln") else 0.0)}
    if op == "pack":
        return st
    mix = case["mix"]
    if mix == "logits":
        st["a"] = normal(T, n)
    elif mix == "matrix":
        st["a"] = normal(n, std=0.1) + 1.0 / n
    else:
        st["a"] = None
    st["g"] = torch.empty(d, device="cuda").uniform_(0.5, 1.5, generator=gen)
    if op in ("ln", "ln_backward"):
        st["beta"] = normal(d, std=0.1)
        if op == "ln_backward":
            st["dx"] = normal(T, d).to(_DT[dt])
            if case["packed"]:
                st["H"] = _pack(st["H"])
        return st
    st["A"] = normal(T, n, n) if mix == "logits" else torch.eye(n, device="cuda") + normal(n, n, std=0.02)
    st["b"] = normal(n, mean=1.0, std=0.02)
    st["y"] = _streams(gen, (T, d), dt)
    st["dHout"] = normal(T, n, d).to(_DT[dt])
    st["dx"] = normal(T, d).to(_DT[dt])
    if op == "backward":
        st["H"] = _pack(st["H"])
        st["y"] = _pack(st["y"])
    return st


# ---- the plain form -------------------------------------------------------------

def _sinkhorn(L):
    """The projection and its 2K + 1 iterates (each iteration needs the one before)."""
    its = [L.exp()]
    for k in range(2 * K):
        its.append(its[-1] / its[-1].sum(-1 - k % 2, keepdim=True))
    return its


def _sinkhorn_backward(its, G):
    for k in reversed(range(2 * K)):
        axis = -1 - k % 2
        G = (G - (G * its[k + 1]).sum(axis, keepdim=True)) / its[k].sum(axis, keepdim=True)
    return G * its[0]


def _softmax(l):
    e = (l - l.amax(-1, keepdim=True)).exp()
    return e / e.sum(-1, keepdim=True)


def _read_weights(st):
    """Per-token read weights [T or 1][n]."""
    if st["case"]["mix"] == "logits":
        return _softmax(st["a"])
    return st["a"][None] if st["a"] is not None else torch.ones(1, 1, device="cuda")


def _read_backward(st, a, da):
    return a * (da - (a * da).sum(-1, keepdim=True)) if st["case"]["mix"] == "logits" else da


def _step_forward(st, H, y, A, a):
    dt = st["H"].dtype
    Hn = (A.transpose(-1, -2) @ H + st["b"][:, None] * y[:, None]).to(dt)
    h = (a[:, :, None] * Hn.float()).sum(1)
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return Hn, (h * r * st["g"]).to(dt)


def _step_backward(st, H, y, A, a, its):
    """Gradients at the values H [T][n][d], y [T][d] (fp32)."""
    dt, b = st["dx"].dtype, st["b"]
    T, n, d = H.shape
    dHn, dx = st["dHout"].float(), st["dx"].float()
    Hn = A.transpose(-1, -2) @ H + b[:, None] * y[:, None]
    h = (a[:, :, None] * Hn).sum(1)
    r = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    u = dx * st["g"]
    dh = r * u - (r ** 3 * (u * h).sum(-1, keepdim=True) / d) * h
    dg = (dx * h * r).sum(0)
    da = (dh[:, None] * Hn).sum(-1)
    G = dHn + a[:, :, None] * dh[:, None]
    dA = H @ G.transpose(-1, -2)
    db = (y[:, None] * G).sum(-1)
    dH = (A @ G).to(dt)
    dy = (b[:, None] * G).sum(1).to(dt)
    if its is not None:
        dA = _sinkhorn_backward(its, dA)
    return {"dH": dH, "dy": dy, "dA": dA, "db": db, "da": _read_backward(st, a, da), "dg": dg}


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "pack":
        return _unpack(*_pack(st["H"])).to(st["H"].dtype)
    a = _read_weights(st)
    if op in ("step", "backward"):
        its = _sinkhorn(st["A"]) if case["mix"] == "logits" else None
        A = its[-1] if its is not None else st["A"]
        if op == "backward":
            return _step_backward(st, _unpack(*st["H"]), _unpack(*st["y"]), A, a, its)
        Hn, x = _step_forward(st, st["H"].float(), st["y"].float(), A, a)
        out = _step_backward(st, _unpack(*_pack(st["H"])), _unpack(*_pack(st["y"])), A, a, its)
        return {"Hout": Hn, "x": x, **out}
    H = _unpack(*st["H"]) if case.get("packed") else st["H"].float()
    h = (a[:, :, None] * H).sum(1)
    h = h - h.mean(-1, keepdim=True)
    rs = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    xh = h * rs
    if op == "ln":
        return (xh * st["g"] + st["beta"]).to(st["H"].dtype)
    dx = st["dx"].float()
    u = dx * st["g"]
    dh = rs * (u - u.mean(-1, keepdim=True) - xh * (u * xh).mean(-1, keepdim=True))
    out = {"dH": (a[:, :, None] * dh[:, None]).to(st["dx"].dtype), "dg": (dx * xh).sum(0), "dbeta": dx.sum(0)}
    if case["mix"] != "none":
        out["da"] = _read_backward(st, a, (dh[:, None] * H).sum(-1))
    return out


# ---- the library's entry points ---------------------------------------------------

def _own(st):
    from hyper_connections_stream_b200 import _lib as hc
    case = st["case"]
    op = case["op"]
    if op == "pack":
        return hc.checkpoint_unpack(hc.checkpoint_pack(st["H"]), st["H"].dtype)
    logits = case["mix"] == "logits"
    read = hc.READ_SOFTMAX_LOGITS if logits else hc.READ_WEIGHTS
    if op == "ln":
        return hc.read_layernorm(st["H"], st["a"], st["g"], st["beta"], eps=EPS, read=read)
    if op == "ln_backward":
        H = hc.Checkpoint(*st["H"]) if case["packed"] else st["H"]
        out = hc.read_layernorm_backward(H, st["a"], st["g"], st["dx"], eps=EPS, read=read)
        return {k: v for k, v in out.items() if v is not None}
    kw = dict(eps=EPS, mix=hc.MIX_SINKHORN_LOGITS if logits else hc.MIX_MATRIX, K=K if logits else 0, read=read)
    if op == "backward":
        return hc.write_then_read_backward_checkpoint(
            hc.Checkpoint(*st["H"]), hc.Checkpoint(*st["y"]), st["A"], st["b"], st["a"], st["g"], st["dHout"],
            st["dx"], **kw)
    Hn, x, cH, cy = hc.write_then_read_checkpoint(st["H"], st["y"], st["A"], st["b"], st["a"], st["g"], **kw)
    out = hc.write_then_read_backward_checkpoint(cH, cy, st["A"], st["b"], st["a"], st["g"], st["dHout"], st["dx"],
                                                 **kw)
    return {"Hout": Hn, "x": x, **out}


def run(state):
    return _own(state) if own else _plain(state)


# ---- fp64 ---------------------------------------------------------------------------

def _pow2(e):
    """2^e in fp64 for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _kept64(x):
    """The values a checkpoint keeps of x, in fp64: every block scaled by its power of two, rounded to 4 significant
    bits (steps of 2^-9 below 2^-6), ties to even."""
    x = x.double()
    d = x.shape[-1]
    pad = -d % BLOCK
    b = torch.nn.functional.pad(x, (0, pad)).reshape(*x.shape[:-1], -1, BLOCK)
    m, e = torch.frexp(b.abs().amax(-1, keepdim=True) / 448.0)       # in [0.5, 1) * 2^e
    e = torch.where(m == 0.5, e - 1, e)
    e = torch.where(m == 0.0, torch.full_like(e, -126), e).clamp(min=-126)
    v = b * _pow2(-e)
    _, ev = torch.frexp(v)
    step = _pow2((ev - 4).clamp(min=-9))
    return (torch.round(v / step) * step * _pow2(e)).reshape(*x.shape[:-1], d + pad)[..., :d]


def _values64(H):
    if isinstance(H, tuple):
        q, s = H
        d = q.shape[-1]
        e = torch.repeat_interleave(s.long() - 127, BLOCK, dim=-1)[..., :d]
        return q.float().double() * _pow2(e)
    return H.double()


def _project64(L):
    M = [torch.exp(L)]
    for _ in range(K):
        M.append(M[-1] / M[-1].sum(dim=-1, keepdim=True))
        M.append(M[-1] / M[-1].sum(dim=-2, keepdim=True))
    return M


def exact(case, seed):
    st = prepare(case, seed)
    T, n, d, op = case["T"], case["n"], case["d"], case["op"]
    logits = case.get("mix") == "logits"
    part = max(1, (1 << 26) // (n * d))
    outs, summed = [], {}
    for t0 in range(0, T, part):
        sl = slice(t0, min(T, t0 + part))

        def cut(v):
            return tuple(w[sl] for w in v) if isinstance(v, tuple) else v[sl]

        H = _values64(cut(st["H"]))
        if op == "pack":
            outs.append({"out": _kept64(H)})
            continue
        m = H.shape[0]
        if st["a"] is None:
            a = torch.ones(m, n, dtype=torch.float64, device="cuda")
        elif logits:
            a = torch.softmax(st["a"][sl].double(), -1)
        else:
            a = st["a"].double().expand(m, n)
        g = st["g"].double()
        if op in ("ln", "ln_backward"):
            h = torch.einsum("tn,tnd->td", a, H)
            mu = h.mean(-1, keepdim=True)
            sd = torch.sqrt(((h - mu) ** 2).mean(-1, keepdim=True) + EPS)
            z = (h - mu) / sd
            if op == "ln":
                outs.append({"out": z * g + st["beta"].double()})
                continue
            dx = st["dx"][sl].double()
            dz = dx * g
            dh = (dz - dz.mean(-1, keepdim=True) - z * (dz * z).mean(-1, keepdim=True)) / sd
            o = {"dH": torch.einsum("tn,td->tnd", a, dh)}
            da = torch.einsum("td,tnd->tn", dh, H)
            sums = {"dg": (dx * z).sum(0), "dbeta": dx.sum(0)}
        else:
            y = _values64(cut(st["y"]))
            b = st["b"].double()
            M = _project64(st["A"][sl].double()) if logits else None
            A = M[-1] if logits else st["A"].double().expand(m, n, n)
            o = {}
            if op == "step":
                Hn = torch.einsum("tij,tid->tjd", A, H) + b[:, None] * y[:, None]
                o["Hout"] = Hn
                h = torch.einsum("tj,tjd->td", a, Hn.to(_DT[case["dt"]]).double())
                o["x"] = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * g
                H, y = _kept64(H), _kept64(y)
            Hn = torch.einsum("tij,tid->tjd", A, H) + b[:, None] * y[:, None]
            h = torch.einsum("tj,tjd->td", a, Hn)
            q = torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
            dx = st["dx"][sl].double()
            dz = dx * g
            dh = dz / q - h * ((dz * h).mean(-1, keepdim=True) / q ** 3)
            G = st["dHout"][sl].double() + a[:, :, None] * dh[:, None]
            da = torch.einsum("td,tjd->tj", dh, Hn)
            dA = torch.einsum("tid,tjd->tij", H, G)
            if logits:
                for k in range(2 * K - 1, -1, -1):
                    axis = -1 if k % 2 == 0 else -2
                    dA = (dA - (dA * M[k + 1]).sum(axis, keepdim=True)) / M[k].sum(axis, keepdim=True)
                dA = dA * M[0]
            o.update(dH=torch.einsum("tij,tjd->tid", A, G), dy=torch.einsum("j,tjd->td", b, G), dA=dA,
                     db=torch.einsum("td,tjd->tj", y, G))
            sums = {"dg": (dx * h / q).sum(0)}
        if st["a"] is not None:
            o["da"] = a * (da - (a * da).sum(-1, keepdim=True)) if logits else da
        outs.append(o)
        summed = {k: summed.get(k, 0.0) + v for k, v in sums.items()}
    cat = {k: torch.cat([o[k] for o in outs]) for k in outs[0]}
    return cat["out"] if "out" in cat else {**cat, **summed}


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    T, n, d, op = case["T"], case["n"], case["d"], case["op"]
    s = 2 if case["dt"] == "bf16" else 4
    q = d + -(-d // BLOCK)               # bytes of one checkpoint row
    logits = case.get("mix") == "logits"
    par = 4 * (n * n + n) if logits else 0      # per-token logits
    if op == "pack":
        # x in, its kept values out, and the checkpoint written and read
        return {"bytes": T * n * (2 * s * d + 2 * q), "flops": T * n * d * 4}
    if op == "ln":
        return {"bytes": T * (s * d * (n + 1) + (4 * n if logits else 0)) + 8 * d, "flops": T * d * (2 * n + 8)}
    if op == "ln_backward":
        src = n * q if case["packed"] else s * n * d
        return {"bytes": T * (src + s * d * (n + 1) + (8 * n if logits else 4 * n)) + 12 * d,
                "flops": T * d * (5 * n + 16)}
    back = T * ((n + 1) * q + 2 * s * (n + 1) * d + par + 4 * (n * n + 2 * n)) + 8 * d
    bflops = T * d * 2 * (2 * n * n + 8 * n + 8)
    if op == "backward":
        return {"bytes": back, "flops": bflops}
    fwd = T * ((n + 1) * q + 2 * s * (n + 1) * d + par) + 4 * d
    return {"bytes": back + fwd, "flops": bflops + T * d * (2 * n * n + 4 * n + 8)}
