"""The build: the library needs nvcc alone; the Python binding follows the
PyTorch that is installed (CPU, on a small source of its own)."""
import os
import shutil
import sys

import pytest

from weight_recurrence_gb300 import build as labuild

pytestmark = pytest.mark.skipif(shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"),
                                reason="no nvcc")


COMMAND = labuild.binding_command


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A package of one small unit, whose binding is 'compiled' by copying its source."""
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (tmp_path / "include").mkdir()
    (tmp_path / "include" / "la.h").write_text("\n")
    (pkg / "csrc" / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (pkg / "csrc" / "la_torch.cpp").write_text("first\n")
    monkeypatch.setattr(labuild, "PKG", str(pkg))
    monkeypatch.setattr(labuild, "CSRC", str(pkg / "csrc"))
    monkeypatch.setattr(labuild, "LIBDIR", str(pkg / "lib"))
    monkeypatch.setattr(labuild, "BINDING_SRC", str(pkg / "csrc" / "la_torch.cpp"))
    monkeypatch.setattr(labuild, "BINDING", str(pkg / "lib" / "_la_torch.so"))
    monkeypatch.setattr(labuild, "binding_command", lambda out: ["cp", str(pkg / "csrc" / "la_torch.cpp"), out])
    return pkg


def test_the_library_builds_without_torch(tree, monkeypatch):
    monkeypatch.setattr(labuild, "binding_command", COMMAND)
    monkeypatch.setattr(labuild.importlib.util, "find_spec", lambda name: None)
    path = labuild.build()
    assert os.path.exists(path) and not os.path.exists(tree / "lib" / "_la_torch.so")


def test_a_binding_that_does_not_compile_leaves_the_library(tree, monkeypatch):
    monkeypatch.setattr(labuild, "binding_command", lambda out: [sys.executable, "-c", "raise SystemExit(1)"])
    with pytest.raises(RuntimeError, match="la_torch.cpp"):
        labuild.build()
    assert os.path.exists(tree / "lib" / "liblinattn.so")


def test_the_binding_follows_its_source_and_the_installed_torch(tree, monkeypatch):
    so = tree / "lib" / "_la_torch.so"
    labuild.build()
    assert so.read_text() == "first\n"
    so.write_text("kept")                       # newer than its source: not made again
    labuild.build()
    assert so.read_text() == "kept"
    monkeypatch.setattr(labuild, "torch_identity", lambda: "another version")
    labuild.build()
    assert so.read_text() == "first\n"
    so.write_text("kept")
    labuild.build()
    assert so.read_text() == "kept"
    monkeypatch.setattr(labuild, "torch_identity", lambda: None)     # PyTorch is gone: nothing to make one for
    labuild.build()
    assert so.read_text() == "kept"


def test_the_identity_names_version_and_place():
    torch = pytest.importorskip("torch")
    text = labuild.torch_identity()
    assert torch.__version__ in text and os.path.dirname(torch.__file__) in text
