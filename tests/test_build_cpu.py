"""The build: the C library does not wait for, or need, PyTorch (the compilers are stood in for), and no C++
exception leaves its C entries."""

import os
import shutil
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


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_no_exception_leaves_a_c_entry(tmp_path):
    here, pkg = os.path.dirname(os.path.abspath(__file__)), os.path.dirname(b.__file__)
    exe = str(tmp_path / "no_throw_check")
    rocm = os.path.dirname(os.path.dirname(b.HIPCC))
    subprocess.run(["g++", "-O1", "-std=c++17", "-D__HIP_PLATFORM_AMD__", f"-I{os.path.join(rocm, 'include')}",
                    f"-I{os.path.join(pkg, 'csrc')}", f"-I{os.path.join(b.ROOT, 'include')}",
                    os.path.join(here, "no_throw_check.cpp"), os.path.join(pkg, "libgemm_bf16.so"), f"-Wl,-rpath,{pkg}",
                    "-Wl,--allow-shlib-undefined", "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout.endswith("ok\n"), r.stdout + r.stderr
