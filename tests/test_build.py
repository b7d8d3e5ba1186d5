"""What the build step builds (no compiler runs): the CUDA library needs nvcc alone,
the extension module belongs to one Python and one torch."""
import importlib.metadata
import importlib.util
import os

import pytest

from fp8_block_scaled_11_b200 import build


@pytest.fixture
def made(monkeypatch):
    """The commands that would run: (compiler, output)."""
    runs = []
    monkeypatch.setattr(build, "_run", lambda cmd, path: runs.append((os.path.basename(cmd[0]), path)))
    monkeypatch.setattr(build, "needs_build", lambda: False)
    monkeypatch.delenv("NVCC", raising=False)
    return runs


def test_without_torch(made, monkeypatch):
    """The C library is for programs without Python and torch too."""
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    assert build.build(force=True) == build.LIB_PATH
    assert made == [("nvcc", build.LIB_PATH)]


def test_torch_without_metadata(made, monkeypatch):
    """A torch that was never installed by a package tool says its version itself."""
    import torch

    def none(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", none)
    build.build(force=True)
    assert torch.__version__ in made[1][1]


def test_with_torch(made):
    build.build(force=True)
    assert [c for c, _ in made] == ["nvcc", "g++"] and made[0][1] == build.LIB_PATH
    assert os.path.basename(made[1][1]).startswith("_binding.") and made[1][1].endswith(".so")


def test_another_torch_has_another_module(made, monkeypatch):
    """A module built for another torch is neither loaded nor taken for up to date."""
    real = importlib.metadata.version
    build.build(force=True)
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.0" if name == "torch" else real(name))
    build.build()
    assert made[2][0] == "g++" and "99.0" in made[2][1] and made[2][1] != made[1][1]
