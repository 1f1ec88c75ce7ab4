"""The package without torch: the library loads, and what needs no tensor runs."""

import os
import subprocess
import sys

from dlrm_embeddings_dot_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import sys
sys.modules["torch"] = None          # any import of it raises
import dlrm_embeddings_dot_gb300 as dl
L = dl.load()
assert (dl.DLRM_ACT_SILU, dl.DLRM_MOE_MAX_TOKENS) == (3, 64)
assert L.dlrm_ws_align(1) == 256
# the dense network's entry points have their signatures: a refusal on the host, by raw addresses
assert L.dlrm_linear_fwd_workspace_size(0x10000, 64, 0x10000, 64, 1, 4096, 512, 64) >= 0
assert L.dlrm_dropout_fwd(None, 8, None, 0, 0, 4, 8, 0.1, None, None, 8, None) == dl.DLRM_ERR_INVALID_ARG
assert "dlrm_dropout_fwd" in dl.dlrm_last_error()
try:
    dl.dlrm_linear_fwd
except ImportError:
    pass
else:
    raise AssertionError("the tensor functions need torch")
print("ok")
"""


def test_library_loads_without_torch():
    libbuild.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
