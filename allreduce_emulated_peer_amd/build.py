"""Build the HIP library libmscl.so in-tree for gfx950.

Two translation units: csrc/mscl.hip (the collectives' C ABI, including the
kernels of csrc/kernels.hpp) and csrc/operators.hip (the linear layer and
layer norm), compiled side by side with hipcc: -O3, no fast-math, no FP
contraction, packed-FP32 instructions disabled.
"""

from __future__ import annotations

import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
SRC = os.path.join(CSRC, "mscl.hip")
UNITS = ("mscl", "operators")
LIB = os.path.join(HERE, "libmscl.so")
ARCH = "gfx950"

FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    "-ffp-contract=off", "-fno-fast-math", "-Wall",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]
# the port channel's proxy drives the SDMA engines through HSA
LIBS = ["-L/opt/rocm/lib", "-lhsa-runtime64"]


def build(verbose: bool = False, extra=(), units=UNITS) -> str:
    """Compile `units` (the others' objects are taken as they are) and link."""
    compiling = []
    for unit in units:
        obj = os.path.join(CSRC, f"{unit}.o")
        cmd = ["/opt/rocm/bin/hipcc", *FLAGS, *extra, "-c", "-o", obj, os.path.join(CSRC, f"{unit}.hip")]
        if verbose:
            print(" ".join(cmd), flush=True)
        compiling.append((cmd, subprocess.Popen(cmd)))
    for cmd, process in compiling:
        if process.wait() != 0:
            raise subprocess.CalledProcessError(process.returncode, cmd)
    tmp = LIB + ".tmp"
    cmd = ["/opt/rocm/bin/hipcc", f"--offload-arch={ARCH}", "-shared", "-o", tmp,
           *[os.path.join(CSRC, f"{unit}.o") for unit in UNITS], *LIBS]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def asm(out_path: str, src: str = SRC) -> str:
    """Device assembly of one translation unit (for inspection)."""
    cmd = ["/opt/rocm/bin/hipcc", *[f for f in FLAGS if f != "-fPIC"], "--cuda-device-only", "-S", "-o", out_path, src]
    subprocess.run(cmd, check=True)
    return out_path


if __name__ == "__main__":
    import sys

    print(build(verbose=True, units=tuple(u for u in sys.argv[1:] if u) if len(sys.argv) > 1 else UNITS))
