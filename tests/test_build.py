"""The CUDA library is built with nvcc alone: the Python binding beside it needs
torch's headers, and its failure does not take the library along."""
from __future__ import annotations

import importlib.util
import os
import shutil

import pytest

from quantized_gguf_dequant_gb300 import build as qbuild

pytestmark = pytest.mark.skipif(
    not os.path.exists(qbuild.nvcc()) and shutil.which("nvcc") is None, reason="nvcc is needed")


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build of one source into a directory of its own."""
    monkeypatch.setattr(qbuild, "SOURCES", ["tmap.cu"])
    monkeypatch.setattr(qbuild, "BUILD", str(tmp_path / "objects"))
    monkeypatch.setattr(qbuild, "LIB", str(tmp_path / "libqmm.so"))
    monkeypatch.setattr(qbuild, "NATIVE", str(tmp_path / "_native.so"))
    return tmp_path


def test_library_without_torch(elsewhere, monkeypatch):
    found = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else found(name, *a))
    assert qbuild.build() == qbuild.LIB
    assert os.path.exists(qbuild.LIB) and not os.path.exists(qbuild.NATIVE)
    made = os.path.getmtime(qbuild.LIB)
    qbuild.build()  # nothing is stale
    assert os.path.getmtime(qbuild.LIB) == made


def test_library_when_the_binding_does_not_compile(elsewhere, monkeypatch):
    pytest.importorskip("torch")
    monkeypatch.setenv("CXX", str(elsewhere / "no-such-compiler"))
    with pytest.raises(RuntimeError, match="binding"):
        qbuild.build()
    assert os.path.exists(qbuild.LIB) and not os.path.exists(qbuild.NATIVE)


def test_binding_alone_when_it_alone_is_stale(elsewhere):
    pytest.importorskip("torch")
    qbuild.build()
    made = os.path.getmtime(qbuild.LIB)
    os.remove(qbuild.NATIVE)
    qbuild.build()
    assert os.path.exists(qbuild.NATIVE) and os.path.getmtime(qbuild.LIB) == made
