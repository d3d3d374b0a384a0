"""Backward calls of no tokens, without a GPU: sums over tokens are outputs all
the same, so an address that cannot hold them is refused, not passed over (fake
device addresses, in a child process that sees no device)."""
from __future__ import annotations

import json
import os
import subprocess
import sys
import textwrap

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

_CHILD = textwrap.dedent(r"""
    import json
    from hyper_connections_stream_b200 import _lib as B
    L = B.lib()
    n, d, at = 4, 1024, 1 << 32
    def step(dg):
        return L.hc_write_then_read_backward_checkpoint(None, None, None, None, B.HC_BF16, 0, n, d, 0, None, 0, 0, None,
                                                        0, 0, None, 0, None, 1e-6, None, None, None, None, None, None,
                                                        None, dg, None, 0, None)
    def norm(dg, dbeta):
        return L.hc_read_layernorm_backward(None, None, B.HC_BF16, 0, n, d, 0, None, 0, None, 1e-6, None, None, None,
                                            dg, dbeta, None, 0, None)
    print(json.dumps([step(None), step(at + 2), norm(None, None), norm(at + 1, None), norm(None, at + 2)]))
""")


def test_misaligned_sums_are_refused():
    from hyper_connections_stream_b200 import build
    build.build()
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    out = subprocess.run([sys.executable, "-c", _CHILD], capture_output=True, text=True, env=env, cwd=ROOT, timeout=300)
    assert out.returncode == 0, out.stderr
    OK, MISALIGNED = 0, 3
    assert json.loads(out.stdout.strip().splitlines()[-1]) == [OK, MISALIGNED, OK, MISALIGNED, MISALIGNED]
