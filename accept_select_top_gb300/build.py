"""Builds libspecdec.so (the verify/accept kernels and their C ABI) for sm_103a.

Each .cu file is compiled by its own nvcc process, in parallel, then linked
into ``_build/libspecdec.so``.  Usage: ``python -m accept_select_top_gb300.build``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libspecdec.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]

# Registers a thread that a kernel has to be launched with: its warp groups trade them, and the split counts
# on what the compiler gives it (a launch with fewer would wait for ever, and is refused).
REGISTERS = {"attention_q8_tc.cu": ("attention_q8_tc_kernel", 80)}


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecdec.so")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return hs


def _stale(obj: str, src: str) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in [src] + _headers())


def check_registers(log: str, kernel: str, want: int) -> None:
    """Raises unless ptxas' report gives every instance of `kernel` `want` registers."""
    got = [int(n) for name, n in re.findall(r"Compiling entry function '(\S+)'.*?Used (\d+) registers", log, re.S)
           if kernel in name]
    if not got or any(n != want for n in got):
        raise RuntimeError(f"{kernel} is written for {want} registers a thread at launch; this compiler gives it {got}: "
                           "its kRegs and the split by role have to follow")


def _compile(src: str, extra) -> str:
    name = os.path.basename(src)
    obj = os.path.join(BUILD, name[:-3] + ".o")
    if _stale(obj, src):
        need = REGISTERS.get(name)
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, *FLAGS, *(["-Xptxas", "-v"] if need else []), *extra, "-c", src, "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {name}:\n{r.stdout}\n{r.stderr}")
        if need:
            check_registers(r.stdout + r.stderr, *need)
        os.replace(tmp, obj)
    return obj


def build(verbose: bool = False, extra=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra)), srcs))
    if not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
