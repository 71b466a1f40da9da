"""Build libtgemm.so in-tree with nvcc for sm_103a (no CMake, a few translation units at once),
and _calls.so, the native calls of the newer operators from torch tensors, with g++."""

from __future__ import annotations

import glob
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libtgemm.so")
CALLS = os.path.join(PKG, "_calls.so")
ARCH = "arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libtgemm needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return all(os.path.getmtime(s) <= t for s in sources())


def nvcc_command(out: str = LIB, extra: list[str] | None = None) -> list[str]:
    return [
        _nvcc(), "-gencode", ARCH, "-O3", "-std=c++17", "-lineinfo",
        "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr",
        "-t", "0", "-I", INCLUDE, "-I", CSRC,
        *(os.path.join(CSRC, f) for f in ("tgemm.cu", "w4.cu", "norm.cu")), "-o", out,
    ] + (extra or [])


def calls_command(out: str = CALLS) -> list[str]:
    import sysconfig
    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return [
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
        "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
        os.path.join(CSRC, "calls.cpp"), "-o", out, "-L", lib, "-Wl,-rpath," + lib,
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
    ]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libtgemm.so and _calls.so next to this file unless newer than every source."""
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    cmd = nvcc_command(tmp, ["-Xptxas", "-v"] if verbose else None)
    calls = calls_command(CALLS + ".tmp")
    other = subprocess.Popen(calls, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    said, _ = other.communicate()
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    if other.returncode != 0:
        raise RuntimeError("g++ failed:\n" + " ".join(calls) + "\n" + said)
    if verbose:
        print(r.stdout + r.stderr)
    os.replace(CALLS + ".tmp", CALLS)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
