"""Runs pieces of host code against the library with a stand-in for the HIP runtime (hip_stand_in.cpp): no GPU is used, no
kernel runs. Each piece is a process of its own, so that the stand-in is what the library binds to."""

from __future__ import annotations

import json
import os
import subprocess
import sys

import persistent_tiled_gemm_amd as ptg

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")

PRELUDE = """
import ctypes, json, sys
sys.path.insert(0, {root!r})
hip = ctypes.CDLL({stand_in!r}, mode=ctypes.RTLD_GLOBAL)
hip.stand_in_launches.restype = hip.stand_in_kernels.restype = ctypes.c_char_p
lib = ctypes.CDLL({library!r})
import persistent_tiled_gemm_amd as ptg
ptg._lib = lib
from persistent_tiled_gemm_amd import layer
layer._lib = None
lib = layer._library()
P = 0x100000  # a made-up, aligned device address
A, B = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x2000)  # two streams
plan = ctypes.c_void_p()

def call(f, args, stream=None):
    return f(ctypes.byref(args), plan, stream)
"""


def built(folder) -> str:
    out = os.path.join(str(folder), "hip_stand_in.so")
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROCM, "include"),
                    os.path.join(HERE, "hip_stand_in.cpp"), "-o", out], check=True)
    return out


def run(stand_in: str, body: str):
    """What the piece `body` leaves in `result`."""
    code = PRELUDE.format(root=ROOT, stand_in=stand_in, library=ptg.LIB_PATH) + body + "\nprint('RESULT ' + json.dumps(result))\n"
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert res.returncode == 0, res.stderr[-4000:]
    return json.loads([x for x in res.stdout.splitlines() if x.startswith("RESULT ")][-1][7:])
