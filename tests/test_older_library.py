"""A library, or a checking extension, of before the residual blocks (include/dlrm_block.h): what it has runs,
what it has not is told of."""

import os
import subprocess
import sys

import pytest

from dlrm_embeddings_dot_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PROGRAM = """
import ctypes, sys, types
import torch
import dlrm_embeddings_dot_gb300 as dl
from dlrm_embeddings_dot_gb300 import block_abi, dense

OLD, NEW = set(block_abi.ENTRY_POINTS + block_abi.SIZES), "{what}"
if NEW == "extension":                      # the library is of before the blocks
    lib = dl.load()
    class Library:
        def __getattr__(self, name):
            if name in OLD:
                raise AttributeError(name)
            return getattr(lib, name)
    dl.load = lambda path=None: Library()
else:                                       # the extension is
    from dlrm_embeddings_dot_gb300 import _marshal as real
    old = types.ModuleType(real.__name__)
    for n in ("bind", "dropout_fwd", "dropout_bwd", "linear_fwd", "linear_bwd", "moe_fwd"):
        setattr(old, n, getattr(real, n))
    sys.modules[real.__name__] = old
    import dlrm_embeddings_dot_gb300 as package
    package._marshal = old

x = torch.zeros(4, 16)
try:                                        # the dense network's calls come as far as their own checks
    dl.dlrm_linear_fwd(x, torch.zeros(8, 16), None, None, torch.zeros(4, 8))
except ValueError as e:
    assert "not on a CUDA device" in str(e), e
u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
calls = [lambda: dl.dlrm_pack8(x, u8(4, 16), u8(4, 1)), lambda: dl.dlrm_unpack8(u8(4, 16), u8(4, 1), x),
         lambda: dl.dlrm_block_norm_fwd(x, None, x, None, None, None, None, None, x, x),
         lambda: dl.dlrm_block_norm_bwd(x, x, x, None, x, torch.zeros(4, 4), *[None] * 12),
         lambda: dl.dlrm_route_fwd(x, i32(4, 2), torch.zeros(4, 2)),
         lambda: dl.dlrm_route_bwd(torch.zeros(4, 2), i32(4, 2), torch.zeros(4, 2), x),
         lambda: dl.dlrm_expert_sort(i32(4, 2), 3, i32(4), i32(4, 2)),
         lambda: dl.dlrm_dispatch_fwd(x, i32(4, 2), x), lambda: dl.dlrm_dispatch_bwd(x, i32(4, 2), x),
         lambda: dl.dlrm_combine_fwd(x, i32(4, 2), torch.zeros(4, 2), None, x),
         lambda: dl.dlrm_combine_bwd(x, x, i32(4, 2), torch.zeros(4, 2), x, None),
         lambda: dl.dlrm_linear_bwd8(x, u8(4, 16), u8(4, 1), torch.zeros(16, 16), None, None, x, None, None)]
if NEW == "extension":
    calls += [lambda: dl.dlrm_block_norm_bwd_workspace_size(x), lambda: dl.dlrm_expert_sort_workspace_size(i32(4, 2), 3),
              lambda: dl.dlrm_linear_bwd8_workspace_size(x, u8(4, 16), torch.zeros(16, 16))]
for call in calls:
    try:
        call()
    except RuntimeError as e:
        assert "build it again" in str(e), e
    else:
        raise AssertionError("ran")
print("ok")
"""


@pytest.mark.parametrize("newer", ["extension", "library"])
def test_what_an_older_build_has_runs(newer):
    libbuild.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM.replace("{what}", newer)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr
