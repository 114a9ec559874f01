"""Builds liblinattn.so in-tree with nvcc for sm_100a.

The library links the CUDA runtime statically and resolves the driver's
tensor-map encoder at run time, so it loads (and exports its symbols) on a
machine without a GPU; only the kernel launches need a B200.

Usage: python -m weight_state_recurrence_b200.build [--force] [--verbose]
"""
from __future__ import annotations

import glob
import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "liblinattn.so")
HEADER = os.path.join(ROOT, "include", "linattn.h")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
]
LINK_FLAGS = ["-shared", "-cudart", "static"]
OBJ = os.path.join(HERE, "_build")


def nvcc() -> str:
    p = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(p):
        raise RuntimeError("nvcc not found")
    return p


def sources():
    """What the library is made from, this file and the flags in it among them."""
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + [HEADER, os.path.abspath(__file__)])


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(s) > t for s in sources())


def _reads(path: str, seen: set) -> set:
    """path and every file it includes by a quoted name."""
    path = os.path.normpath(path)
    if path not in seen:
        seen.add(path)
        with open(path) as f:
            for name in re.findall(r'^#include "([^"]+)"', f.read(), re.M):
                _reads(os.path.join(os.path.dirname(path), name), seen)
    return seen


def _compile(src: str, force: bool, verbose: bool) -> str:
    """One translation unit to its object file, unless that is newer than all it reads and than
    the flags in this file."""
    obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
    if force or not os.path.exists(obj) or any(
            os.path.getmtime(p) > os.path.getmtime(obj)
            for p in {os.path.abspath(__file__), *_reads(src, set())}):
        tmp = f"{obj}.tmp{os.getpid()}.o"
        subprocess.check_call([nvcc(), *NVCC_FLAGS, *(["-Xptxas", "-v"] if verbose else []),
                               "-c", "-o", tmp, src])
        os.replace(tmp, obj)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with ThreadPoolExecutor(len(units)) as pool:   # nvcc processes, side by side
        objs = list(pool.map(lambda u: _compile(u, force, verbose), units))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([nvcc(), *NVCC_FLAGS, *LINK_FLAGS, "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="--verbose" in sys.argv)
    print(LIB)
