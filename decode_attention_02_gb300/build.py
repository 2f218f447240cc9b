"""Compile libmfa.so (the CUDA kernels and the C ABI) in-tree for sm_103a."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libmfa.so")
SOURCES = [os.path.join(PKG, "csrc", f) for f in
           ("mfa_decode.cu", "mfa_kv_append.cu", "mfa_block_decode.cu", "mfa_block_append.cu", "mfa_rope.cu")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (CUDA toolkit required to build libmfa.so)")
    return cand


def _inputs():
    return (SOURCES + glob.glob(os.path.join(PKG, "csrc", "*.cuh")) + glob.glob(os.path.join(PKG, "csrc", "*.h")) +
            [os.path.join(ROOT, "include", "mfa.h")])


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _inputs())


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Build libmfa.so next to this file; returns its path."""
    if not force and not needs_build():
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    flags = [*ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
             "-I" + os.path.join(ROOT, "include"), *extra_flags]
    if verbose:
        flags.insert(0, "-Xptxas=-v")
        print(" ".join(flags))
    # one compiler process per source, side by side; then the link
    objects = [f"{tmp}.{i}.o" for i in range(len(SOURCES))]
    jobs = [subprocess.Popen([_nvcc(), *flags, "-c", "-o", obj, src]) for src, obj in zip(SOURCES, objects)]
    try:
        failed = [src for src, job in zip(SOURCES, jobs) if job.wait() != 0]
        if failed:
            raise RuntimeError("nvcc failed on " + ", ".join(failed))
        subprocess.check_call([_nvcc(), *ARCH, "-shared", "-o", tmp, *objects])
    finally:
        for obj in objects:
            if os.path.exists(obj):
                os.remove(obj)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose="-v" in sys.argv))
