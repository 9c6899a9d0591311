"""Compile libmoe_amd.so for gfx950 with hipcc, and the compiled Python calls for this
interpreter and torch with the host compiler (in-tree, no JIT cache).  Both are put in
place together, so that calls of another build never meet the library's descriptors."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe_amd.so")

SOURCES = ["route.hip", "align.hip", "layout.hip", "experts.hip", "gemm.hip",
           "few.hip", "fp8_gemm.hip", "quant.hip", "mxfp4.hip", "mxfp4_gemm.hip", "norm.hip",
           "moe_api.cpp"]
HEADERS = ["moe_common.h", "moe_gemm_tile.h", "moe_kernels.h"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-Wall", "-Wno-unused-function",
    # never let the compiler form packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found: the HIP library cannot be built")
    return p


def _run(cmd, verbose: bool, noise: str = ""):
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if not noise or noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({r.returncode}):\n{err}")
    if verbose and err.strip():
        print(err)


def calls_path() -> str:
    """Of the compiled calls for this interpreter and this torch: a file for others is not
    taken for them."""
    import torch
    return os.path.join(LIBDIR, f"_moe_calls.{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def calls_lack() -> str:
    """What the compiled calls need and is not here ("": nothing)."""
    if host_cxx() is None:
        return "a host C++ compiler"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python's headers"
    import torch
    return "" if os.path.isdir(os.path.join(os.path.dirname(torch.__file__), "include")) else "torch's headers"


def host_cxx():
    return shutil.which("g++") or shutil.which("c++") or shutil.which("amdclang++", path=os.path.dirname(hipcc()))


def _compile_calls(to: str, verbose: bool):
    import torch
    base = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(base, "include"), os.path.join(base, "lib")
    _run([host_cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"),
          os.path.join(CSRC, "calls.cpp"), "-o", to, "-L", lib, f"-Wl,-rpath,{lib}",
          "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose)


def _compile_library(to: str, verbose: bool):
    srcs = []
    for s in SOURCES:
        path = os.path.join(CSRC, s)
        # .cpp sources also hold HIP runtime calls: compile all as HIP
        srcs += ["-x", "hip", path]
    cmd = [hipcc()] + HIPCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC] + srcs + ["-o", to]
    _run(cmd, verbose, noise="is not a recognized feature for this target")


def build(verbose: bool = False) -> str:
    """The library, and the calls where what they need is here (else a warning: the 4-bit
    operators and the norm are then without Python calls, the others are whole)."""
    os.makedirs(LIBDIR, exist_ok=True)
    lib, calls = LIB + ".tmp", None
    _compile_library(lib, verbose)
    if lack := calls_lack():
        warnings.warn(f"no Python calls of the 4-bit operators and the norm: {lack} is not here")
    else:
        calls = calls_path()
        _compile_calls(calls + ".tmp", verbose)
    os.replace(lib, LIB)
    for name in os.listdir(LIBDIR):   # (calls for this library alone)
        if name.startswith("_moe_calls") and name.endswith(".so"):
            os.remove(os.path.join(LIBDIR, name))
    if calls:
        os.replace(calls + ".tmp", calls)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
