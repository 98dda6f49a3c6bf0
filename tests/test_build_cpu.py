"""The build's order: the C library does not wait for, or need, PyTorch. The compilers are stood in for."""

import os
import subprocess
import sys

import pytest

from gemv_layers_amd import build as b


@pytest.fixture
def made(monkeypatch, tmp_path):
    """Every output in tmp_path, made by a stand-in that writes its -o file; returns their names in order."""
    names = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        with open(out, "w") as f:
            f.write("built")
        names.append(os.path.basename(out).split(".tmp")[0])
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libgemm_bf16.so"))
    monkeypatch.setattr(b, "TORCH_OUT", str(tmp_path / "_torch_ops.so"))
    return names


def test_the_library_builds_without_pytorch(made, monkeypatch, tmp_path, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)              # import torch fails
    monkeypatch.setitem(sys.modules, "torch.utils.cpp_extension", None)
    assert b.build() == str(tmp_path / "libgemm_bf16.so")
    assert "libgemm_bf16.so" in made and "_torch_ops.so" not in made
    assert (tmp_path / "libgemm_bf16.so").exists() and "PyTorch" in capsys.readouterr().err


def test_a_module_that_does_not_compile_leaves_a_library(made, monkeypatch, tmp_path):
    def fails():
        raise RuntimeError("torch_ops.cpp failed")

    monkeypatch.setattr(b, "_build_torch_ops", fails)
    with pytest.raises(RuntimeError, match="torch_ops"):
        b.build()
    assert (tmp_path / "libgemm_bf16.so").exists()
