"""Build libnvfp4hs.so in-tree with nvcc for sm_100a (no JIT cache)."""
from __future__ import annotations

import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnvfp4hs.so")
# the checked build: bounds checks on every global access of the per-step
# kernels and the K/V cache's (-DNVFP4HS_CHECKS), for debugging and for the
# edge-case tests
LIB_CHECKED = os.path.join(PKG, "libnvfp4hs_checked.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-shared", "-Xcompiler", "-fPIC",
    "-t", "0",  # the sources are compiled side by side
    # IEEE division/sqrt and denormals stay on (nvcc defaults); no fast-math.
]


# GEMMs (X^T X and GPTQ's batch updates) and the Cholesky factorizations of
# the GPTQ path come from cuBLAS and cuSOLVER
LIBS = ["-lcublas", "-lcusolver"]


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, checked: bool = False) -> str:
    lib = LIB_CHECKED if checked else LIB
    if not force and not _stale(lib):
        return lib
    nvcc = os.environ.get("NVCC", "nvcc")
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc, *NVCC_FLAGS, *(["-DNVFP4HS_CHECKS"] if checked else []), "-I", INCLUDE, "-I",
           CSRC, *sources(), *LIBS, "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    subprocess.check_call(cmd)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
