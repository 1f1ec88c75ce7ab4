"""Build the CUDA library ``libdlrm_gb300.so`` (sm_103a) in the package directory.

Each ``csrc/*.cu`` (and host-only ``csrc/*.cpp``) file is compiled by nvcc
in parallel and linked into one shared object exporting the C ABI of
``include/*.h``.  The CUDA runtime is linked statically, so the
library needs only the driver at run time.  ``csrc/marshal.c`` becomes the
small CPython extension ``_marshal`` beside it, which the dense network's
tensor functions need; where there is no C compiler or no Python headers the
library is built all the same.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdlrm_gb300.so")
MARSHAL_SRC = os.path.join(CSRC, "marshal.c")
# the dense network's argument checks, a CPython extension: its name carries the Python version it is for
MARSHAL = os.path.join(HERE, "_marshal" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _digest(files, flags) -> str:
    h = hashlib.sha256()
    for f in files:
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(flags).encode())
    return h.hexdigest()


def _up_to_date(out: str, stamp: str, digest: str) -> bool:
    if not (os.path.exists(out) and os.path.exists(stamp)):
        return False
    with open(stamp) as f:
        return f.read() == digest


def _write(stamp: str, digest: str) -> None:
    with open(stamp, "w") as f:
        f.write(digest)


def _library_digest() -> str:
    files = _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]
    return _digest(files, ARCH + FLAGS)


def _build_marshal(force: bool) -> None:
    """Compiles the extension unless an up-to-date one exists; a failure is a warning, and the tensor
    functions that need it raise when they are called."""
    include = sysconfig.get_paths()["include"]
    digest = _digest(sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [MARSHAL_SRC, os.path.abspath(__file__)],
                     [sys.version, include])
    stamp = os.path.join(BUILD, os.path.basename(MARSHAL) + ".stamp")
    if not force and _up_to_date(MARSHAL, stamp, digest):
        return
    cc = shutil.which("gcc") or shutil.which("cc")
    tmp = MARSHAL + f".{os.getpid()}.tmp"
    why = "no C compiler"
    if cc:
        try:
            r = subprocess.run([cc, "-O2", "-shared", "-fPIC", "-I", include, "-I", INCLUDE, "-o", tmp, MARSHAL_SRC],
                               capture_output=True, text=True)
            why = f"{r.stdout}\n{r.stderr}".strip() if r.returncode else ""
        except OSError as e:
            why = str(e)
    if why:
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)        # it is for other sources
        warnings.warn(f"{os.path.basename(MARSHAL)} was not built, so the dense network's tensor functions will not run "
                      f"(it needs a C compiler and Python's headers): {why}", RuntimeWarning, stacklevel=3)
        return
    os.replace(tmp, MARSHAL)
    _write(stamp, digest)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link the library, and the extension, unless up-to-date builds exist."""
    os.makedirs(BUILD, exist_ok=True)
    stamp = os.path.join(BUILD, "stamp")
    digest = _library_digest()
    if force or not _up_to_date(LIB, stamp, digest):
        _build_library(verbose)
        _write(stamp, digest)
    _build_marshal(force)
    return LIB


def _build_library(verbose: bool) -> None:
    nvcc = _nvcc()

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD, os.path.splitext(os.path.basename(src))[0] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".{os.getpid()}.tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
