"""Build the HIP library in-tree: hipcc for gfx950 -> fully_sharded_amd/libfsdp_mi355x.so.

Run ``python -m fully_sharded_amd._build`` (or ``__graft_entry__.build()``).
It compiles every time it is called.
"""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfsdp_mi355x.so")
SOURCES = ["plan.cpp", "kernels.hip", "abi.cpp", "graph.cpp", "muon.hip", "muon.cpp"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# IEEE fp32: correctly rounded divide and sqrt, denormals kept, no fast-math,
# no implicit FMA contraction (the kernels write their FMAs explicitly), and
# no packed-fp32 instructions.  Kernel arguments preloaded into scalar
# registers at wave launch (gfx950 supports up to 16): a workgroup then
# reads its work descriptor without first loading the table's address from
# the argument segment, one memory round trip fewer before its first data
# load.  The code object keeps the argument loads as a fallback for a
# command processor that does not preload.  Measured on MI355X, alternating
# runs: the 12-layer model's step 383.5 -> 381.5 us, its standalone fused
# step 23.3 -> 23.1 us.
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-ffp-contract=off",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-Wall",
]


def build(verbose: bool = True) -> str:
    objs = []
    os.makedirs(os.path.join(PKG, "_build"), exist_ok=True)
    for src in SOURCES:
        obj = os.path.join(PKG, "_build", src + ".o")
        cmd = [HIPCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd[1:1] = ["-x", "hip"]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp,
           "-Wl,-rpath,/opt/rocm/lib", "-Wl,--no-undefined"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    build_c_driver(verbose)
    return LIB


# A plain C99 program that drives one training step through the C ABI with
# device memory from the HIP runtime (tests/c/step_from_c.c): the GPU tests
# run it to show the library works without Python.  Host code only (gcc).
C_DRIVER_SRC = os.path.join(ROOT, "tests", "c", "step_from_c.c")
C_DRIVER = os.path.join(ROOT, "tests", "c", "step_from_c")


def build_c_driver(verbose: bool = True) -> str:
    tmp = C_DRIVER + ".tmp"
    cmd = ["gcc", "-std=c99", "-O2", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE,
           "-I", "/opt/rocm/include", C_DRIVER_SRC, "-o", tmp, "-L", PKG, "-lfsdp_mi355x",
           "-L", "/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,$ORIGIN/../../fully_sharded_amd",
           "-Wl,-rpath,/opt/rocm/lib"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, C_DRIVER)
    return C_DRIVER


if __name__ == "__main__":
    build(verbose="-q" not in sys.argv)
