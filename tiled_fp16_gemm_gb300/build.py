"""Build libtgemm.so in-tree with nvcc for sm_103a (no CMake, a few translation units at once),
and, where PyTorch with CUDA is installed, _calls.so, the native calls of the newer operators
from torch tensors, with g++.  The C library needs neither PyTorch nor _calls.so."""

from __future__ import annotations

import glob
import importlib.util
import os
import runpy
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


def _torch() -> tuple[str, str] | None:
    """Folder and version of the installed PyTorch, if it is one with CUDA (not imported here)."""
    try:
        spec = importlib.util.find_spec("torch")
    except (ImportError, ValueError):
        return None
    if spec is None or not spec.submodule_search_locations:
        return None
    where = list(spec.submodule_search_locations)[0]
    about = runpy.run_path(os.path.join(where, "version.py"))
    return (where, str(about["__version__"])) if about.get("cuda") else None


def _mark(torch: tuple[str, str]) -> str:
    """What _calls.so says of the PyTorch that it was built against (its ABI differs by version)."""
    return "built against torch " + torch[1]


def _newer(made: str) -> bool:
    t = os.path.getmtime(made) if os.path.exists(made) else -1.0
    return all(os.path.getmtime(s) <= t for s in sources())


def _calls_current() -> bool:
    torch = _torch()
    if torch is None:
        return True  # nothing to build
    if not _newer(CALLS):
        return False
    with open(CALLS, "rb") as f:
        return _mark(torch).encode() + b"\0" in f.read()


def up_to_date() -> bool:
    return _newer(LIB) and _calls_current()


def nvcc_command(out: str = LIB, extra: list[str] | None = None) -> list[str]:
    return [
        _nvcc(), "-gencode", ARCH, "-O3", "-std=c++17", "-lineinfo",
        "-Xcompiler", "-fPIC", "-shared", "--expt-relaxed-constexpr",
        "-t", "0", "-I", INCLUDE, "-I", CSRC,
        *(os.path.join(CSRC, f) for f in ("tgemm.cu", "w4.cu", "norm.cu", "layer_norm.cu", "i8.cu")), "-o", out,
    ] + (extra or [])


def calls_command(out: str = CALLS) -> list[str]:
    import sysconfig
    torch = _torch()
    inc, lib = os.path.join(torch[0], "include"), os.path.join(torch[0], "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    return [
        "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
        f'-DTG_BUILT_AGAINST="{_mark(torch)}"',
        "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
        "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"),
        os.path.join(CSRC, "calls.cpp"), "-o", out, "-L", lib, "-Wl,-rpath," + lib,
        "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
    ]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libtgemm.so and _calls.so next to this file unless newer than every source (and
    _calls.so built against another PyTorch).  A library that compiled is kept whatever becomes
    of the other."""
    other = None
    if force or not _calls_current():
        if _torch() is not None:
            calls = calls_command(CALLS + ".tmp")
            try:
                other = subprocess.Popen(calls, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
            except OSError as e:
                other = e
    said = ""
    if force or not _newer(LIB):
        tmp = LIB + ".tmp"
        cmd = nvcc_command(tmp, ["-Xptxas", "-v"] if verbose else None)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode == 0:
            os.replace(tmp, LIB)
            if verbose:
                print(r.stdout + r.stderr)
        else:
            said = "nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr
    if isinstance(other, OSError):
        said += f"g++ failed:\n{other}"
    elif other is not None:
        out, _ = other.communicate()
        if other.returncode == 0:
            os.replace(CALLS + ".tmp", CALLS)
        else:
            said += "g++ failed:\n" + " ".join(calls) + "\n" + out
    if said:
        raise RuntimeError(said)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
