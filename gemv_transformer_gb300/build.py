"""Build libwq.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each ``csrc/*.cu`` is compiled in parallel to an object, then linked into
``gemv_transformer_gb300/_build/libwq.so`` with the static CUDA runtime.  ``py_calls.c``, the
binding's marshalling of the decode-step calls, is compiled with gcc beside it where gcc and
Python's headers are there; the library does not need it, and the binding does without.
Run ``python -m gemv_transformer_gb300.build`` or call :func:`build`.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.machinery
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB = os.path.join(OUT_DIR, "libwq.so")
# Named for the interpreter that it is built for: another one builds its own.
CALLS = os.path.join(OUT_DIR, "_wq_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])
CALLS_SRC = os.path.join(CSRC, "py_calls.c")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libwq")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + _headers()


def _newer(path, deps) -> bool:
    return os.path.exists(path) and \
        all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps + [__file__])


def _can_build_calls() -> bool:
    return shutil.which("gcc") is not None and \
        os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def _calls_up_to_date() -> bool:
    return not _can_build_calls() or _newer(CALLS, [CALLS_SRC] + _headers())


def up_to_date() -> bool:
    return _newer(LIB, _deps()) and _calls_up_to_date()


def _build_calls():
    tmp = CALLS + f".{os.getpid()}.tmp"
    cmd = ["gcc", "-O2", "-std=gnu11", "-shared", "-fPIC", "-I",
           sysconfig.get_paths()["include"], "-o", tmp, CALLS_SRC]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on {CALLS_SRC}:\n{r.stderr}")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every kernel for sm_103a and link libwq.so; returns its path."""
    os.makedirs(OUT_DIR, exist_ok=True)
    if force or not _newer(LIB, _deps()):
        _build_lib(verbose, ptxas_info)
    if not _can_build_calls():
        sys.stderr.write("py_calls.c: no gcc or no Python.h, the binding will use ctypes alone\n")
    elif force or not _calls_up_to_date():
        _build_calls()
    return LIB


def _build_lib(verbose: bool, ptxas_info: bool) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
