"""Build the HIP library libtp1proj.so in-tree for gfx950.

The library is the C ABI of include/tp1_proj.h: host plan logic (plan.cpp,
tactics_table.cpp), the ABI (proj_abi.hip) and the kernels (kernels.hip), and
the layer operators: the norm and row codes (norm.hip), the 8-bit projection
(proj_i8.hip) and the gated delta rule (delta_*.hip).
All HIP code is compiled with packed-FP32 instructions disabled.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
LIB = os.path.join(PKG, "libtp1proj.so")
ARCH = os.environ.get("TP1_OFFLOAD_ARCH", "gfx950")

SOURCES = ["plan.cpp", "tactics_table.cpp", "proj_abi.hip", "kernels.hip", "probes.hip",
           "norm.hip", "proj_i8.hip", "delta_abi.hip", "delta_step.hip", "delta_chunk.hip"]

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    f"--offload-arch={ARCH}",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    f"-I{os.path.join(ROOT, 'include')}",
]


def hipcc() -> str:
    path = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(path):
        raise RuntimeError("hipcc not found: the HIP library cannot be built")
    return path


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every source and link libtp1proj.so; returns its path."""
    out_dir = os.path.join(PKG, "_build")
    os.makedirs(out_dir, exist_ok=True)
    objs = []
    for src in SOURCES:
        obj = os.path.join(out_dir, os.path.splitext(src)[0] + ".o")
        cmd = [hipcc(), *HIPCC_FLAGS, *(extra or []), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if src.endswith(".cpp"):
            cmd.insert(1, "-x")
            cmd.insert(2, "c++")
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
