"""Compile libmoe_amd.so for gfx950 with hipcc, and the compiled Python calls for this
interpreter and torch with the host compiler (in-tree, no JIT cache)."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libmoe_amd.so")
CALLS = os.path.join(LIBDIR, "_moe_calls.so")

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


def build_calls(verbose: bool = False) -> str:
    import torch
    base = os.path.dirname(torch.__file__)
    inc, lib = os.path.join(base, "include"), os.path.join(base, "lib")
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("no host C++ compiler: the Python calls cannot be built")
    tmp = CALLS + ".tmp"
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-I", os.path.join(ROOT, "include"),
          os.path.join(CSRC, "calls.cpp"), "-o", tmp, "-L", lib, f"-Wl,-rpath,{lib}",
          "-ltorch_python", "-ltorch_cpu", "-lc10"], verbose)
    os.replace(tmp, CALLS)
    return CALLS


def build(verbose: bool = False) -> str:
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = []
    for s in SOURCES:
        path = os.path.join(CSRC, s)
        # .cpp sources also hold HIP runtime calls: compile all as HIP
        srcs += ["-x", "hip", path]
    tmp = LIB + ".tmp"
    cmd = [hipcc()] + HIPCC_FLAGS + ["-I", os.path.join(ROOT, "include"), "-I", CSRC] + srcs + ["-o", tmp]
    _run(cmd, verbose, noise="is not a recognized feature for this target")
    os.replace(tmp, LIB)
    build_calls(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
