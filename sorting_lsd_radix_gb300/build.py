"""Builds the gbsort CUDA library (libgbsort.so) in the package directory.

Each .cu file is compiled for sm_103a in parallel, then linked into one shared
library with the CUDA runtime linked statically.  No CMake.  Beside it,
_rows.*.so is the row operators' calls from Python (rows_py.c, plain C), where
Python's headers and a C compiler are installed; without it the binding calls
through ctypes."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgbsort.so")
# with the interpreter's tag: another version of Python does not import it
ROWS_PY = os.path.join(PKG, "_rows" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
SOURCES = ["api.cu", "radix.cu", "radix_wide.cu", "radix11.cu", "bitonic.cu", "noalloc.cu", "expert.cu",
           "embedding.cu", "id_order.cu", "rows_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _flags(extra=()):
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                   "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")] + list(extra)


def _deps_mtime():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(ROOT, "include", f) for f in os.listdir(os.path.join(ROOT, "include"))]
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def _build_rows_py():
    include = sysconfig.get_paths()["include"]
    gcc = os.environ.get("CC") or "gcc"
    if not os.path.exists(os.path.join(include, "Python.h")) or shutil.which(gcc) is None:
        return
    tmp = ROWS_PY + f".tmp{os.getpid()}"
    cmd = [gcc, "-O2", "-Wall", "-shared", "-fPIC", "-I", include, "-I",
           os.path.join(ROOT, "include"), os.path.join(CSRC, "rows_py.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on rows_py.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, ROWS_PY)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        if not os.path.exists(ROWS_PY):
            _build_rows_py()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc] + _flags(extra_flags) + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        rows_py = ex.submit(_build_rows_py)
        objs = list(ex.map(compile_one, SOURCES))
        rows_py.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
