"""The build where the dense network's extension cannot be compiled."""

import os
import subprocess
import sys

import pytest

from dlrm_embeddings_dot_gb300 import build as libbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def no_compiler(monkeypatch, tmp_path):
    """A tree whose library is up to date and whose extension is not, on a machine without Python's headers."""
    libbuild.build()
    fake = tmp_path / "gcc"
    fake.write_text("#!/bin/sh\necho 'Python.h: No such file or directory' >&2\nexit 1\n")
    fake.chmod(0o755)
    which = libbuild.shutil.which
    monkeypatch.setattr(libbuild.shutil, "which", lambda n, *a, **k: str(fake) if n in ("gcc", "cc") else which(n, *a, **k))
    monkeypatch.setattr(libbuild, "MARSHAL", str(tmp_path / os.path.basename(libbuild.MARSHAL)))
    return monkeypatch


def test_library_is_built_without_the_extension(no_compiler):
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert libbuild.build() == libbuild.LIB
    assert not os.path.exists(libbuild.MARSHAL)
    # the library counts as built: another call compiles nothing
    no_compiler.setattr(libbuild, "_nvcc", lambda: pytest.fail("the library was compiled again"))
    with pytest.warns(RuntimeWarning):
        libbuild.build()
    no_compiler.setattr(libbuild.shutil, "which", lambda *a, **k: None)
    with pytest.warns(RuntimeWarning, match="no C compiler"):
        libbuild.build()


def test_extension_is_named_after_its_python():
    assert os.path.basename(libbuild.MARSHAL).startswith("_marshal.") and libbuild.MARSHAL.endswith(
        libbuild.sysconfig.get_config_var("EXT_SUFFIX"))


def test_tensor_functions_say_what_is_missing():
    """Without the extension the dense network's functions raise when called; the rest of the package works."""
    program = """
import sys
sys.modules["dlrm_embeddings_dot_gb300._marshal"] = None
import torch, dlrm_embeddings_dot_gb300 as dl
dl.load()
x = torch.zeros(2, 2)
try:
    dl.dlrm_dropout_fwd(x, None, x, 0.0, None)
except RuntimeError as e:
    assert "_marshal" in str(e)
    print("ok")
"""
    r = subprocess.run([sys.executable, "-c", program], cwd=ROOT, capture_output=True, text=True)
    assert r.stdout.strip() == "ok", r.stderr
