"""Pieces of a summed index hold each element once (k_piece_check.cpp, on the kernels' own function)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host C++ compiler")
def test_pieces_hold_each_element_once(tmp_path):
    exe = str(tmp_path / "k_piece_check")
    csrc = os.path.join(os.path.dirname(HERE), "gemv_layers_amd", "csrc")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", f"-I{csrc}", os.path.join(HERE, "k_piece_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
