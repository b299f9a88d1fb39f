"""Build libgfr.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import os
import subprocess
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgfr.so")
SOURCES = [os.path.join(CSRC, f) for f in (
    "gfr_kernels.hip", "gfr_api.cpp", "gfr_linear.hip", "gfr_moe_decode.hip",
    "gfr_moe_route.hip", "gfr_layer_api.cpp")]

HIPCC_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # never emit packed-FP32 VALU ops
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
]


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source (side by side), link, and replace the library."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.check_call(cmd)

    with tempfile.TemporaryDirectory() as tmp:
        objects = [os.path.join(tmp, os.path.basename(s) + ".o") for s in SOURCES]
        with ThreadPoolExecutor(4) as pool:
            list(pool.map(lambda so: run([hipcc, *HIPCC_FLAGS, *extra_flags, "-I", INCLUDE, "-I",
                                          CSRC, "-c", so[0], "-o", so[1]]),
                          zip(SOURCES, objects)))
        out = LIB + ".tmp"
        run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *objects, "-o", out])
    os.replace(out, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
