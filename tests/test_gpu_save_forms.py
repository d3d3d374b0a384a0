"""The step that keeps a checkpoint in every form its launch can choose: the
register-streaming family, and the pipelined family with its default consumer
groups and with the eight-warp groups that rows take which pad the default more
(bf16 d = 4096, fp32 d = 2048, up to four streams). Whatever the form, H' and x
are write_then_read's and the checkpoints checkpoint_pack's, bit for bit."""
from __future__ import annotations

import pytest
import torch

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
    L.set_path(L.PATH_AUTO)
    yield L
    L.set_path(L.PATH_AUTO)
    torch.cuda.synchronize()
    assert L.device_fault() == 0


def _normal(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda") * std + mean


def _check(hc, path, T, n, d, dt, logits):
    H, y = _normal(21, T, n, d).to(DT[dt]), _normal(22, T, d).to(DT[dt])
    H[0, 0, d - 1] = float("nan")
    y[T - 1, 0] = float("-inf")
    lead = (T,) if logits else ()
    A = _normal(23, *lead, n, n) if logits else torch.eye(n, device="cuda") + _normal(23, n, n, std=0.3)
    a, b, g = _normal(24, *lead, n), _normal(25, n, mean=1.0, std=0.2), _normal(26, d, mean=1.0, std=0.2)
    kw = dict(eps=EPS, mix=int(logits), K=20 if logits else 0, read=int(logits))
    hc.set_path(hc.PATH_AUTO)
    want = hc.write_then_read(H, y, A, b, a, g, **kw)
    wH, wy, nb = hc.checkpoint_pack(H), hc.checkpoint_pack(y), -(-d // 32)
    hc.set_path(path)
    bits = lambda t: t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)
    for out in (None, H.clone()):
        src = H if out is None else out
        Hn, x, cH, cy = hc.write_then_read_checkpoint(src, y, A, b, a, g, out=out, **kw)
        for got, ref in ((Hn, want[0]), (x, want[1])):
            nan = ref.isnan()
            assert torch.equal(got.isnan(), nan)
            assert torch.equal(bits(got)[~nan], bits(ref)[~nan])
        for c, w in ((cH, wH), (cy, wy)):
            assert torch.equal(c.codes.view(torch.uint8), w.codes.view(torch.uint8))
            assert torch.equal(c.scales[..., :nb], w.scales[..., :nb])


# pipelined: enough tokens that CTAs take several; rows of one tile, of whole
# tiles, and that end inside one
@pytest.mark.parametrize("logits", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,slices", [(1, 224), (1, 512), (2, 448), (2, 512), (3, 300), (3, 512), (4, 448), (4, 512),
                                      (4, 131), (5, 256), (5, 193), (6, 320), (7, 130), (8, 256), (8, 67)])
def test_pipelined(hc, n, slices, dt, logits):
    _check(hc, hc.PATH_PIPELINED, 700, n, slices * (8 if dt == "bf16" else 4), dt, logits)


@pytest.mark.parametrize("T,n,d,dt", [(4096, 4, 4096, "bf16"), (9000, 3, 4096, "bf16"), (1300, 3, 2048, "f32")])
def test_eight_warp_groups_where_the_rule_takes_them(hc, T, n, d, dt):
    """The static layer's size, and sizes on either side of the 8192 tokens that
    bound the fused step's eight-warp groups (not this step's)."""
    for path in (hc.PATH_AUTO, hc.PATH_PIPELINED):
        _check(hc, path, T, n, d, dt, False)


@pytest.mark.parametrize("logits", [True, False])
@pytest.mark.parametrize("n,d,dt", [(1, 512, "bf16"), (2, 1032, "bf16"), (4, 4096, "f32"), (5, 1544, "bf16"),
                                    (6, 8192, "bf16"), (7, 16384, "f32"), (8, 520, "bf16"), (8, 4096, "bf16"),
                                    (8, 32768, "bf16")])
def test_register_streaming(hc, n, d, dt, logits):
    _check(hc, hc.PATH_REGISTER, 310 if d < 16384 else 40, n, d, dt, logits)
