"""Builds libdsa.so (the C-ABI library of include/dsa.h) in-tree with nvcc for sm_103a.

Each .cu file under csrc/ compiles in parallel to an object under _build/,
then nvcc links them into two_tier_sparse_gb300/libdsa.so. The binding's own compiled part
(csrc/calls.c, a CPython module) goes to two_tier_sparse_gb300/_calls.<tag>.so where the Python
headers are there, and is left out elsewhere. No CMake.
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

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdsa.so")
# (the interpreter's tag in its name: a module of one Python is not for another)
CALLS = os.path.join(PKG, "_calls" + importlib.machinery.EXTENSION_SUFFIXES[0])

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr"]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _stale(obj: str, deps: list[str]) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                     + glob.glob(os.path.join(ROOT, "include", "*.h")))
    nvcc = _nvcc()
    flags = FLAGS + (extra_flags or [])
    jobs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc, *ARCH, *flags, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    def run(cmd):
        p = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, p

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, p in ex.map(run, jobs):
            if verbose or p.returncode != 0:
                sys.stderr.write(p.stdout + p.stderr)
            if p.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    build_calls(force)
    return LIB


def build_calls(force: bool = False) -> str | None:
    """The binding's compiled part. The library does not need it, and the binding works without
    it: with no Python headers or no gcc it is left out (None), and an old one removed."""
    src = os.path.join(CSRC, "calls.c")
    if force or _stale(CALLS, [src, os.path.join(ROOT, "include", "dsa.h")]):
        include = sysconfig.get_paths()["include"]
        if not os.path.exists(os.path.join(include, "Python.h")) or shutil.which("gcc") is None:
            sys.stderr.write(f"csrc/calls.c is left out: it needs gcc and {include}/Python.h\n")
            if os.path.exists(CALLS):
                os.remove(CALLS)
            return None
        tmp = CALLS + f".tmp{os.getpid()}"
        subprocess.check_call(["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + include,
                               "-I" + os.path.join(ROOT, "include"), src, "-o", tmp])
        os.replace(tmp, CALLS)
    return CALLS


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
