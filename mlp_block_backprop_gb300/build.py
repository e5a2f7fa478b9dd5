"""Builds libmlpblk.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each translation unit compiles in its own nvcc process, in parallel; the objects
are then linked into one shared library next to this file.  No cmake, no torch
extension machinery: the library has a plain C ABI (include/mlpblk.h).
"""

from __future__ import annotations

import glob
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmlpblk.so")
# csrc/pycalls.c: CPython entry to the latency-bound calls, for this interpreter alone
CALLS = os.path.join(HERE, "_mlpblk_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])
SOURCES = ["api.cu", "gemm_fwd.cu", "gemm_bwd.cu", "rowops.cu", "simt_f32.cu", "noalloc.cu", "optim.cu", "fp8.cu", "gemm_f8.cu", "moe.cu",
           "sort.cu", "fp4.cu", "gemm_f4.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-Xptxas", "-v"]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmlpblk.so")
    return path


def _newest_input_mtime() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    paths.append(os.path.join(os.path.dirname(HERE), "include", "mlpblk.h"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def up_to_date(path: str) -> bool:
    return os.path.exists(path) and os.path.getmtime(path) >= _newest_input_mtime()


def _python_headers():
    """The directory of Python.h, or None: without it the binding makes every call
    through ctypes."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) else None


def _build_calls() -> None:
    """csrc/pycalls.c against the library just linked (found beside it at run time)."""
    inc = _python_headers()
    if inc is None:
        return
    tmp = CALLS + ".tmp"
    cmd = [shutil.which("gcc") or "cc", "-O2", "-shared", "-fPIC", "-Wall", "-I", inc, os.path.join(CSRC, "pycalls.c"), "-o", tmp,
           "-L", HERE, "-l:libmlpblk.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"pycalls.c failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def _remove_calls() -> None:
    """Every interpreter's module: they were built against the library before this one."""
    for path in glob.glob(os.path.join(glob.escape(HERE), "_mlpblk_calls*.so")):
        os.remove(path)


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libmlpblk.so; returns its path.  Raises on failure."""
    if not force and up_to_date(LIB):
        if _python_headers() and not up_to_date(CALLS):  # another interpreter than the last one's
            _build_calls()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        return src, obj, r

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    for src, _, r in results:
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
    tmp = LIB + ".tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *[obj for _, obj, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _remove_calls()
    _build_calls()
    return LIB


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
