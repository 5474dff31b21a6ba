"""The build's two outputs: the library does not need the native marshalling, and the marshalling is of one torch."""
from __future__ import annotations

import os

import pytest
import torch

from linear_cross_entropy_tmem_gb300 import binding, build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one empty translation unit into a folder of its own."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "out" / "libflce.so"))
    monkeypatch.setattr(build, "SOURCES", ["one.cu"])
    monkeypatch.setattr(binding, "LIB_PATH", build.LIB)
    return src


def test_library_is_linked_where_the_marshalling_does_not_compile(small):
    (small / build.TORCH_SOURCE).write_text("#error no torch here\n")
    with pytest.raises(RuntimeError, match="no torch here"):
        build.build()
    assert os.path.exists(build.LIB)
    at = os.path.getmtime(build.LIB)
    with pytest.raises(RuntimeError, match="no torch here"):
        build.build()  # raised until it compiles; the library stays
    assert os.path.getmtime(build.LIB) == at


def test_another_torch_gets_a_marshalling_of_its_own(small, monkeypatch):
    (small / build.TORCH_SOURCE).write_text("int two() { return 2; }\n")
    build.build()
    assert torch.__version__ in os.path.basename(binding.torch_path()) and os.path.exists(binding.torch_path())
    monkeypatch.setattr(torch, "__version__", "0.0.0+other")
    monkeypatch.setattr(binding, "_TORCH", None)
    monkeypatch.setattr(binding, "load", lambda: None)
    with pytest.raises(RuntimeError, match="not found"):
        binding.load_torch()
    build.build()
    assert os.path.exists(binding.torch_path())
