"""Build the HIP library libptg_gemm.so in-tree for gfx950 with hipcc.

Usage: python -m persistent_tiled_gemm_amd.build  (or build() from Python).
"""

from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO, "include")
JOBS = 4  # compilers at a time
LIB_NAME = "libptg_gemm.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)

SOURCES = ["gemm_kernel.hip", "spoiler.hip", "mfma_probe.hip", "hbm_probe.hip", "gemm_api.hip",
           "layer_api.hip", "norm_kernel.hip", "act_kernel.hip", "product_kernel.hip", "rows_kernel.hip"]

# gfx950 only. Packed-fp32 VALU forms are disabled (hipcc makes them from plain
# float code; some of their forms have produced wrong results on this part).
HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
    "-Wno-unused-command-line-argument",
]


def hipcc() -> str:
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cand = os.path.join(rocm, "bin", "hipcc")
    return cand if os.path.exists(cand) else "hipcc"


def build(verbose: bool = False) -> str:
    """Compile every HIP source into LIB_PATH; return its path. Always rebuilds."""
    tmp = LIB_PATH + ".tmp"
    flags = [*HIPCC_FLAGS, "-I", INCLUDE, "-I", CSRC]
    # the host pass does not know the packed-fp32 target feature; that warning is harmless
    noise = "'-packed-fp32-ops' is not a recognized feature"

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)

    with tempfile.TemporaryDirectory(prefix="ptg_build_") as objs, ThreadPoolExecutor(JOBS) as pool:
        out = {s: os.path.join(objs, s + ".o") for s in SOURCES}
        # one compiler per source, a few at a time, then one link
        list(pool.map(lambda s: run([hipcc(), *(f for f in flags if f != "-shared"), "-c", os.path.join(CSRC, s), "-o", out[s]]),
                      SOURCES))
        run([hipcc(), *HIPCC_FLAGS, *out.values(), "-o", tmp])
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
