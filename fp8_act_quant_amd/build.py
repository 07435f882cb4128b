"""Build libfp8q.so (the HIP kernels and the C ABI) in-tree for gfx950 with hipcc, and _native.so,
the Python binding of the routed-expert, 8-bit and dense-block operators, against it and torch."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfp8q.so")
BINDING = os.path.join(PKG, "_native.so")

SOURCES = ["api.hip", "quant.hip", "gemm.hip", "transpose.hip", "bf16_gemm.hip", "route.hip", "place.hip",
           "int8.hip", "norm.hip", "gated.hip", "adapter.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # every fp32 rounding is written out explicitly (fmaf where a fused op is wanted)
    "-ffp-contract=off",
    # keep the compiler from forming packed-fp32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # MFMA results in VGPRs: the per-slice promotion FMAs read them directly
    "-mllvm", "-amdgpu-mfma-vgpr-form",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found; ROCm is required to build libfp8q.so")
    return p


def _run(cmd, what, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(what)


def build(verbose: bool = False) -> str:
    """Each source by a compiler of its own, side by side, then the library from them."""
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects, ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
        objs = [os.path.join(objects, s + ".o") for s in SOURCES]
        jobs = [pool.submit(_run, [hipcc(), *HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", o],
                            f"hipcc failed building {s}", verbose) for s, o in zip(SOURCES, objs)]
        for j in jobs:
            j.result()
        _run([hipcc(), "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs], "hipcc failed linking libfp8q.so", verbose)
    os.replace(tmp, LIB)
    build_binding(verbose)
    return LIB


def build_binding(verbose: bool = False) -> str:
    """_native.so: host code only. It finds libfp8q.so beside itself; torch's libraries are loaded
    by the `import torch` before it."""
    import torch
    top = os.path.dirname(torch.__file__)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipcc())))
    cxx = shutil.which("g++")
    if cxx is None:
        raise RuntimeError("g++ not found; it is required to build _native.so")
    tmp = BINDING + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f for d in (os.path.join(top, "include"), os.path.join(rocm, "include"),
                         sysconfig.get_paths()["include"]) for f in ("-isystem", d)),
           "-I", INCLUDE, os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(top, "lib"), "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python",
           "-L", PKG, "-l:libfp8q.so", "-Wl,-rpath,$ORIGIN"]
    _run(cmd, "g++ failed building _native.so", verbose)
    os.replace(tmp, BINDING)
    return BINDING


if __name__ == "__main__":
    print(build(verbose=True))
