"""Build libfp8bs.so in-tree with nvcc for sm_103a.

Each translation unit in csrc/ is compiled in parallel, then linked into one
shared library with the shared CUDA runtime (the same libcudart PyTorch loads,
so streams handed over from torch are valid here).
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libfp8bs.so")
# the same library with the fused kernel's per-phase timeline compiled in
# (-DFP8BS_TRACE, fp8bs_trace_read); a profiling aid, never the default
TRACE_LIB_PATH = os.path.join(BUILD_DIR, "libfp8bs_trace.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["api.cu", "quant.cu", "prepack.cu", "gemm_fused.cu", "rmsnorm_quant.cu", "moe.cu",
           "w4_quant.cu", "w4_gemv.cu", "w4_moe.cu", "moe_route.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return cand


def _inputs() -> list[str]:
    files = [os.path.join(CSRC, s) for s in SOURCES]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    files.append(os.path.join(INCLUDE, "fp8bs.h"))
    return files


def _stale(lib_path: str) -> bool:
    if not os.path.exists(lib_path):
        return True
    t = os.path.getmtime(lib_path)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build(force: bool = False, verbose: bool = False, trace: bool = False) -> str:
    """Compile (if stale) and return the path of libfp8bs.so (trace=True:
    libfp8bs_trace.so, the same sources with FP8BS_TRACE defined)."""
    lib_path = TRACE_LIB_PATH if trace else LIB_PATH
    if not force and not _stale(lib_path):
        return lib_path
    obj_dir = os.path.join(BUILD_DIR, "trace") if trace else BUILD_DIR
    os.makedirs(obj_dir, exist_ok=True)
    nvcc = _nvcc()
    defs = ["-DFP8BS_TRACE"] if trace else []

    def compile_one(src: str) -> str:
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *defs, "-I", INCLUDE, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, trace="--trace" in sys.argv))
