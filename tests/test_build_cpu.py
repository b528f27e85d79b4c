"""What a build needs: the library and its C ABI nvcc alone, the calls with tensors PyTorch and g++."""
import os

import pytest

from dense_linear_projection_gb300 import _build


@pytest.fixture
def commands(monkeypatch):
    """Runs no compiler: records its commands."""
    seen = []
    monkeypatch.setattr(_build, "_run", lambda cmd, what: seen.append(cmd))
    monkeypatch.setattr(_build.os, "replace", lambda a, b: seen.append(["replace", b]))
    return seen


def test_the_library_builds_without_pytorch_and_gxx(commands, monkeypatch):
    def missing(*a, **k):
        raise RuntimeError("PyTorch not found")

    monkeypatch.setattr(_build, "_torch_dir", missing)
    if hasattr(_build, "bind_path"):
        monkeypatch.setattr(_build, "bind_path", lambda: os.path.join(_build.PKG, "no such _bind.so"))
    monkeypatch.setattr(_build.shutil, "which", lambda name, *a: None if name == "g++" else "/usr/local/cuda/bin/" + name)
    assert _build.build(force=True) == _build.library_path()
    assert ["replace", _build.library_path()] in commands
    assert all("nvcc" in c[0] for c in commands if c[0] != "replace")


def test_one_bind_for_each_python_and_pytorch(monkeypatch):
    import torch
    here = _build.bind_path()
    assert os.path.dirname(here) == _build.PKG and here.endswith(".so")
    monkeypatch.setattr(torch, "__version__", "1.0")
    other = _build.bind_path()
    monkeypatch.undo()
    monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-399-none")
    assert len({here, other, _build.bind_path()}) == 3


def test_bind_is_compiled_and_linked_to_the_library(commands, monkeypatch):
    monkeypatch.setattr(_build, "_stale", lambda target, deps: "_bind" in os.path.basename(target))
    assert _build.build_bind() == _build.bind_path()
    assert len(commands) == 3 and commands[-1] == ["replace", _build.bind_path()]
    assert "-l:" + os.path.basename(_build.library_path()) in commands[1]
