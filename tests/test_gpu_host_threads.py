"""Entry points called from several host threads at once. A kernel's largest
dynamic shared memory is a setting of the process: no call may lower what
another one, just before its launch, relies on. A launch that asks for more
than the setting is refused by the runtime (HC_ERR_CUDA) and nothing runs.

The calls are made ready first (arguments of the C entries, outputs held), and
each thread then makes its own one after the other on a stream of its own, with
next to nothing between them that holds the interpreter: the C calls overlap
nearly all the time."""
from __future__ import annotations

import ctypes
import os
import subprocess
import sys
import textwrap
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, F32 = torch.bfloat16, torch.float32


class _Recorder:
    """Stands for the library: keeps the arguments of the entry point called
    (all but the stream, its last), answers workspace queries as it does."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_bytes") or name == "hc_last_error":
            return getattr(self.lib, name)

        def record(*args):
            self.calls.append((getattr(self.lib, name), args[:-1]))
            return 0
        return record


def ready(hc, call):
    """(entry point, its arguments, what they point to) of one binding call."""
    lib, rec = hc.lib(), _Recorder(hc.lib())
    hc.lib = lambda: rec
    try:
        held = call()
    finally:
        hc.lib = lambda: lib
    (fn, args), = rec.calls
    return fn, args, held


def together(hc, lists, times=1):
    """Every list of ready calls in a thread and on a stream of its own, `times`
    times over; returns the errors."""
    torch.cuda.synchronize()  # the inputs are there
    errors, gate = [], threading.Barrier(len(lists))

    def work(calls):
        torch.cuda.init()
        stream = torch.cuda.Stream()
        s = stream.cuda_stream
        gate.wait()
        for _ in range(times):
            for fn, args, _ in calls:
                if fn(*args, s) != 0:
                    errors.append(hc.lib().hc_last_error().decode())
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(c,)) for c in lists]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return sorted(set(errors))


def normal(*s):
    return torch.randn(*s, device="cuda")


def step(hc, T, n, d, K, dt=BF):
    H, y, dx = normal(T, n, d).to(dt), normal(T, d).to(dt), normal(T, d).to(dt)
    return H, y, normal(T, n, n), normal(n), normal(T, n), normal(d), dx, dict(mix=1, K=K, read=1)


def packed_backward(hc, T, n, d, K):
    H, y, A, b, a, g, dx, kw = step(hc, T, n, d, K)
    cH, cy = hc.checkpoint_pack(H), hc.checkpoint_pack(y)

    def call():
        return hc.write_then_read_backward_checkpoint(cH, cy, A, b, a, g, None, dx, **kw), (cH, cy, A, b, a, g, dx)
    return ready(hc, call)


def full_backward(hc, T, n, d, K):
    H, y, A, b, a, g, dx, kw = step(hc, T, n, d, K)

    def call():
        return hc.write_then_read_backward(H, y, A, b, a, g, None, dx, **kw), (H, y, A, b, a, g, dx)
    return ready(hc, call)


def saving_step(hc, n, d, dt):
    H, y, A, b, a, g, _, kw = step(hc, 2, n, d, 2, dt)

    def call():
        return hc.write_then_read_checkpoint(H, y, A, b, a, g, **kw), (H, y, A, b, a, g)
    return ready(hc, call)


def layernorm_backward(hc, n, d, dt, packed):
    H, dx, a, g = normal(2, n, d).to(dt), normal(2, d).to(dt), normal(2, n), normal(d)
    src = hc.checkpoint_pack(H) if packed else H

    def call():
        return hc.read_layernorm_backward(src, a, g, dx, read=1, want_dg=False, want_dbeta=False), (src, dx, a, g)
    return ready(hc, call)


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


def test_parameter_backward_of_few_and_many_iterations(hc):
    """The Sinkhorn backward keeps 2 K + 1 iterates: calls with K = 2 beside
    calls with K = 90, from the checkpoint and in full precision."""
    for make in (packed_backward, full_backward):
        lists = [[make(hc, 6, 4, 64, K)] for K in (2, 90, 2, 90)]
        assert together(hc, lists, 2000) == []


def test_backward_of_short_and_long_rows(hc):
    """The backward parks a row in shared memory: short rows beside long ones."""
    lists = [[full_backward(hc, 2, 2, d, 2)] for d in (64, 16384, 64, 16384)]
    assert together(hc, lists, 2000) == []


_CHILD = textwrap.dedent(r"""
    import sys
    import torch
    from hyper_connections_stream_b200 import _lib as hc
    from tests.test_gpu_host_threads import BF, F32, layernorm_backward, saving_step, together
    which = sys.argv[1]
    hc.set_path(hc.PATH_PIPELINED)
    bad = []
    for dt in (BF, F32):
        v = 8 if dt == BF else 4
        for n in range(1, 9):
            if which == "step":
                rows = [saving_step(hc, n, d, dt) for d in range(2 * v, 250 * v, 4 * v)]
                bad += together(hc, [rows] * 4) + together(hc, [rows[::-1]])
            else:
                for packed in (False, True):
                    rows = [layernorm_backward(hc, n, d, dt, packed) for d in range(16, 1000, 16)]
                    bad += together(hc, [rows] * 4) + together(hc, [rows[::-1]])
    print("\n".join(bad))
    sys.exit(1 if bad else 0)
""")


@pytest.mark.parametrize("which", ["step", "layernorm"])
def test_longer_and_longer_rows_in_a_fresh_process(hc, which):
    """Kernels whose shared memory goes by the row's length, from their first
    call on: four threads with rows of more and more columns, so that one or
    another is always making the longest call so far, then all lengths again.
    (The threads share their outputs; nothing reads them.)"""
    out = subprocess.run([sys.executable, "-c", _CHILD, which], capture_output=True, text=True, cwd=ROOT, timeout=300,
                         env=dict(os.environ, PYTHONPATH=ROOT))
    assert out.returncode == 0, (out.stdout[-2000:], out.stderr[-2000:])


def test_first_call_of_a_host_thread(hc):
    """Entry points that make a driver call (tensor maps; a buffer's range), from
    threads that have made no CUDA call before."""
    H, W, X, Wo = normal(37, 4, 64).to(BF), normal(24, 256).to(BF), normal(37, 64).to(BF), normal(64, 64).to(BF)
    A, b = normal(4, 4), normal(4)
    calls = [lambda: hc.mix_logits(H, W), lambda: hc.linear_then_write(X, Wo, H, A, b)]
    want = [c() for c in calls]
    s = torch.cuda.current_stream().cuda_stream
    for call, ref in zip(calls, want):
        fn, args, res = ready(hc, call)
        got = []
        t = threading.Thread(target=lambda: got.append((fn(*args, s), hc.lib().hc_last_error().decode())))
        t.start()
        t.join()
        torch.cuda.synchronize()
        assert got == [(0, "")]
        assert torch.equal(res, ref)
    buf, got = normal(1 << 20), []
    handle, offset = ctypes.create_string_buffer(64), ctypes.c_uint64(0)
    t = threading.Thread(target=lambda: got.append(hc.lib().hc_ipc_export(buf.data_ptr(), handle, ctypes.byref(offset))))
    t.start()
    t.join()
    assert got == [0]


def test_mixing_logits_of_few_and_many_columns(hc):
    """The tensor-core logits' stages go by P."""
    def make(P):
        H, W = normal(2, 4, 64).to(BF), normal(P, 256).to(BF)
        return ready(hc, lambda: (hc.mix_logits(H, W), H, W))
    rows = [make(P) for P in range(8, 129, 8)]
    assert together(hc, [rows] * 4, 200) == []
