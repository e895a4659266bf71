"""Build libsolattn.so (sm_100a) in-tree with nvcc.

    python -m block_sparse_online_b200.build [--verbose] [--debug]

The library is written next to this file so that it travels with the source
tree; the Python binding loads it from there.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libsolattn.so")
# The same library with the kernels' device-side bounds checks compiled in (-DSOLATTN_DEBUG):
# a failed check records SOLATTN_EBOUNDS in the workspace status word instead of touching
# memory out of range. Same exports; load it explicitly (solattn.load_library(DEBUG_LIB)).
DEBUG_LIB = os.path.join(PKG, "libsolattn_debug.so")
SOURCES = ["solattn_api.cu", "dense_api.cu"]
# The short call path of the binding (host code only).
FASTCALL = os.path.join(PKG, "_fastcall.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def build(verbose: bool = False, extra=(), debug: bool = False) -> str:
    out = DEBUG_LIB if debug else LIB
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--threads", str(len(SOURCES)), "-shared", "-Xcompiler", "-fPIC",
           "-I", INCLUDE, "-I", CSRC, "-o", out, *[os.path.join(CSRC, s) for s in SOURCES], *extra]
    if debug:
        cmd.insert(1, "-DSOLATTN_DEBUG")
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    if verbose:
        sys.stdout.write(res.stdout + res.stderr)
    return out


def build_fastcall() -> str:
    """Compile the binding's short call path against the installed torch."""
    import sysconfig

    from torch.utils import cpp_extension as ext
    inc = [f"-I{p}" for p in ext.include_paths("cuda") + [sysconfig.get_paths()["include"], INCLUDE]]
    lib = [x for p in ext.library_paths("cpu") for x in (f"-L{p}", f"-Wl,-rpath,{p}")]
    import torch
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, "-o", FASTCALL,
           os.path.join(CSRC, "fastcall.cpp"), *lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed:\n" + res.stdout + res.stderr)
    return FASTCALL


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, debug="--debug" in sys.argv))
    if "--debug" not in sys.argv:
        print(build_fastcall())
