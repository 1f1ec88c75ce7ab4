"""The table of the runtime's answers about kernels (csrc/memo.h), on the host: each kernel has its
own answer, in whatever order they are asked for."""

import ctypes
import itertools
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = r"""
#include "memo.h"
using dlrm::KernelMemo;
static int asked;
void first(int) {}
void second(int) {}      // the same type
extern "C" {
KernelMemo* create() { return new KernelMemo; }
void destroy(KernelMemo* m) { delete m; }
int asks() { return asked; }
// the answer is made of the key; which: 0 or 1
int get(KernelMemo* m, int which, int device, int cluster, size_t smem)
{
    const void* k = reinterpret_cast<const void*>(which ? second : first);
    return m->get({k, device, cluster, smem}, [&] { ++asked; return 1000000 * which + 10000 * device + 1000 * cluster + (int)(smem % 997); });
}
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("memo")
    (d / "m.cpp").write_text(SOURCE)
    # -O0: the two empty kernels must not become one
    subprocess.run([shutil.which("g++") or "c++", "-O0", "-std=c++17", "-shared", "-fPIC", "-pthread", "-I",
                    os.path.join(ROOT, "dlrm_embeddings_dot_gb300", "csrc"), "-o", str(d / "m.so"), str(d / "m.cpp")], check=True)
    L = ctypes.CDLL(str(d / "m.so"))
    L.create.restype = ctypes.c_void_p
    L.destroy.argtypes = [ctypes.c_void_p]
    L.get.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_size_t]
    return L


def _answer(which, device, cluster, smem):
    return 1000000 * which + 10000 * device + 1000 * cluster + smem % 997


KEYS = [(w, d, c, s) for w in (0, 1) for d in (0, 1) for c in (2, 4) for s in (172160,)]


def test_answers_do_not_depend_on_the_order(lib):
    for order in itertools.islice(itertools.permutations(KEYS), 0, 40320, 997):
        m = lib.create()
        before = lib.asks()
        for _ in range(2):
            assert [lib.get(m, *k) for k in order] == [_answer(*k) for k in order]
        assert lib.asks() - before == len(KEYS)      # kept from the first time
        lib.destroy(m)


def test_more_answers_than_places(lib):
    m = lib.create()
    for s, w in list(itertools.product(range(0, 128 * 3000, 128), (0, 1))) * 2:
        assert lib.get(m, w, 0, 2, s) == _answer(w, 0, 2, s)
    lib.destroy(m)
