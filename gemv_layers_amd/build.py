"""Build the gfx950 library libgemm_bf16.so in-tree with hipcc (no GPU needed to compile), and the module
that hands PyTorch tensors to it."""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libgemm_bf16.so")
TORCH_OUT = os.path.join(HERE, "_torch_ops.so")
BUILD = os.path.join(ROOT, "_build")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

SOURCES = ["gemm_tile.hip", "gemm_skinny.hip", "gemm_generic.hip", "gemm_mx.hip", "gemm_packed.hip",
           "ops_tile.hip", "i8_decode.hip", "ops_generic.hip", "ops_rows.hip", "group_tile.hip", "f8_tile.hip", "f8_decode.hip", "group_generic.hip", "f8_rows.hip",
           "peak.hip", "plan.cpp", "abi.cpp", "ops.cpp", "ops_grouped.cpp"]

COMMON = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    # no packed-fp32 instructions in device code (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
    f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [HIPCC, *COMMON, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_torch_ops() -> str:
    """The tensor marshalling module: host C++ against the installed PyTorch's headers and libraries."""
    from torch.utils.cpp_extension import include_paths, library_paths

    tmp = TORCH_OUT + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "-no-hip-rt", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-I{os.path.join(ROOT, 'include')}", f"-I{sysconfig.get_paths()['include']}",
           *(f"-isystem{p}" for p in include_paths()), os.path.join(CSRC, "torch_ops.cpp"), "-o", tmp,
           *(f"-L{p}" for p in library_paths()), "-ltorch_python", "-ltorch_cpu", "-lc10_hip", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"torch_ops.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_OUT)
    return TORCH_OUT


def build(jobs: int | None = None) -> str:
    """Compile every source and link libgemm_bf16.so next to this file, then _torch_ops.so where PyTorch
    is installed (the library needs none). Always recompiles."""
    os.makedirs(BUILD, exist_ok=True)
    jobs = jobs or min(len(SOURCES), max(1, min(16, len(os.sched_getaffinity(0)))))
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        torch_ops = ex.submit(_build_torch_ops) if importlib.util.find_spec("torch") else None
        objs = list(ex.map(_compile, SOURCES))
        tmp = OUT + ".tmp%d" % os.getpid()
        cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, OUT)
        if torch_ops:
            torch_ops.result()
        else:
            print("PyTorch is not installed: _torch_ops.so, the 8-bit and training helpers' module, is not built",
                  file=sys.stderr)
    return OUT


if __name__ == "__main__":
    print(build(int(sys.argv[1]) if len(sys.argv) > 1 else None))
