"""What the binding needs to be imported and called with pointers (no GPU)."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import sys
sys.modules["torch"] = None   # any import of it fails
from top_sparse_mla_gb300 import build, native
build()
p = native.dsa_params_init(4, 64, 640, 128, 1000, 1000)
assert native.dsa_sparse_attn_workspace_size(p, 152) > 0
try:
    # a call with pointers and a stream of the caller's own; the first pointer is null
    native.dsa_sparse_attn_fwd(None, 256, 256, 256, 256, 256, 256, 256, 256, p, 256, workspace_bytes=1 << 40, stream=0)
except native.DsaError as e:
    assert e.code == native.DSA_ERR_INVALID_ARG, e
else:
    raise AssertionError("a null pointer was accepted")
"""


def test_pointers_and_a_stream_need_no_torch():
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stderr[-2000:]
