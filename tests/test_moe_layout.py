"""The mixture's dynamic shared memory (csrc/moe_layout.h), checked on the host: what the kernels
use lies within what their launches ask for, wherever the static arrays in front of it end."""

import ctypes
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "moe_layout.h"
using namespace dlrm::moe;
extern "C" {
size_t up_asked(int T, int E, int rings) { return asked(up_used(T, E, rings)); }
size_t down_asked(int T, int rings) { return asked(down_used(T, rings)); }
size_t start(size_t raw) { return area(raw); }
}
"""
WARPS, RING, PITCH, MOST = 8, 8 * 2 * 8192, 20, 232448   # the kernels' own figures; 227 KB a block


@pytest.fixture(scope="module")
def layout(tmp_path_factory):
    d = tmp_path_factory.mktemp("layout")
    (d / "l.cpp").write_text(SOURCE)
    subprocess.run([shutil.which("g++") or "c++", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dlrm_embeddings_dot_gb300", "csrc"), "-o", str(d / "l.so"), str(d / "l.cpp")], check=True)
    lib = ctypes.CDLL(str(d / "l.so"))
    for f in (lib.up_asked, lib.down_asked, lib.start):
        f.restype = ctypes.c_size_t
    lib.start.argtypes = [ctypes.c_size_t]
    return lib


@pytest.mark.parametrize("rings", [0, 1])
def test_shared_memory_covers_what_the_kernels_use(layout, rings):
    # the most that rounding the base up can cost, over every place the static arrays can end
    shift = max(layout.start(raw) - raw for raw in range(4096))
    assert all(layout.start(raw) % 128 == 0 for raw in range(0, 4096, 16))
    for T in range(1, 65):
        sums = WARPS * T * PITCH * 4
        asked = layout.down_asked(T, rings)
        assert shift + (RING if rings else 0) + sums <= asked <= MOST
        tiles = WARPS * 2 * (8 if T <= 8 else 16 if T <= 16 else 32) * PITCH * 4
        for E in range(1, 257):
            e_tiles = -(-E // 16)
            sub = max(1, WARPS // e_tiles)
            logits = (sub + 1) * T * e_tiles * 16 * 4      # partial ones of each split, then the sums
            if rings:
                assert logits <= RING
            used = RING + tiles if rings else max(logits, tiles)
            assert shift + used <= layout.up_asked(T, E, rings) <= MOST
