"""Which kernels the int8 product, the cross entropy, its gradient and the quantiser launch, seen by a stand-in for the HIP
runtime (no GPU)."""

import pytest

from tests import head_cases, hip_stand_in


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return hip_stand_in.built(tmp_path_factory.mktemp("stand_in"))


def test_the_compared_calls_are_what_they_say(stand_in):
    cases = [c[1:] for c in head_cases.CASES]
    got = hip_stand_in.run(stand_in, head_cases.WHAT_RUNS + f"result = [what_runs(*c) for c in {cases!r}]")
    assert {f"{c[1:]}": g for c, g in zip(head_cases.CASES, got)} == {f"{c[1:]}": c[0] for c in head_cases.CASES}


def test_no_call_of_the_range_runs_otherwise(stand_in):
    """Calls over the range that the operators are used in: each launches what the compared ones cover."""
    got = hip_stand_in.run(stand_in, head_cases.WHAT_RUNS + r"""
import math, random
rng = random.Random(11)
def size(lo, hi, step):
    return max(step, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step)
result = {}
for _ in range(30000):
    kind = rng.choice(["i8", "i8", "loss", "dx", "dw"])
    i8 = kind == "i8"
    m, n, k = size(1, 16384, 1), size(64, 17000 if i8 else 140000, 8), size(64, 17000 if i8 else 8300, 16 if i8 else 8)
    if rng.random() < 0.4:
        n, k = (n + 63) // 64 * 64, (k + 127) // 128 * 128
    if m * n * k <= (8192 ** 3 if i8 else 4096 * 4096 * 131072):
        for part in what_runs(kind, m, n, k).split("; "):
            result.setdefault(part, [kind, m, n, k])
""")
    covered = {part for c in head_cases.CASES for part in c[0].split("; ")}
    assert len(got) > 50 and not set(got) - covered, {w: got[w] for w in set(got) - covered}


def test_every_new_kernel_is_launched_by_some_call(stand_in):
    cases = [c[1:] for c in head_cases.CASES]
    got = hip_stand_in.run(stand_in, head_cases.WHAT_RUNS.replace("    words = []\n", "    global seen\n    words = []\n").replace(
        "        name, gx, gy, block, first, chunks = line.split()\n", "        name, gx, gy, block, first, chunks = line.split()\n        seen.add(name)\n") + f"""
seen = set()
for c in {cases!r}:
    what_runs(*c)
for n in (8, 520, 1032, 2056, 4104, 8200, 16392, 32776):
    for t in (0, 1):
        for o in (2, 3):
            a = layer.QuantizeArgs(x=P, out=P, scale=P, m=4, n=n, ldx=n, ldo=n, type=t, out_type=o)
            assert lib.layer_quantize(ctypes.byref(a), None) == 0
        if n <= 32768:
            a = layer.RmsnormArgs(x=P, out=P, scale=P, m=4, n=n, ldx=n, ldo=n, type=t, out_type=3, eps=1e-6)
            assert lib.layer_rmsnorm(ctypes.byref(a), None) == 0
seen |= {{line.split()[0] for line in hip.stand_in_launches().decode().splitlines()}}
result = dict(seen=sorted(seen), kernels=hip.stand_in_kernels().decode().split())
""")
    new = {k for k in got["kernels"] if any(w in k for w in ("_i8_", "ptg_loss", "_loss_kernel", "product_scaled", "ptg_quantise"))}
    assert len(new) > 60 and not new - set(got["seen"]), sorted(new - set(got["seen"]))


def test_super_tiles_visit_every_tile_once(tmp_path):
    """The order that the new products' tiles are walked in, compiled for the host."""
    import ctypes
    import os
    import re
    import subprocess

    csrc = os.path.join(hip_stand_in.ROOT, "persistent_tiled_gemm_amd", "csrc")
    text = open(os.path.join(csrc, "ptg_device.hpp")).read()
    body = re.search(r"__device__ __forceinline__ void decode_super_tile\(.*?\n}\n", text, re.S).group(0)
    src = tmp_path / "decode.cpp"
    src.write_text("#include <stdint.h>\n#include <algorithm>\nusing std::min;\nstatic constexpr int kXcdRegions = 8;\n"
                   + body.replace("__device__ __forceinline__", "static")
                   + '\nextern "C" int at(int t, int tm, int tn, int g) { int m, n; decode_super_tile(t, tm, tn, g, m, n); return m * 100000 + n; }\n')
    subprocess.run(["g++", "-O2", "-shared", "-fPIC", str(src), "-o", str(tmp_path / "decode.so")], check=True)
    at = ctypes.CDLL(str(tmp_path / "decode.so")).at
    for tm in (1, 2, 3, 7, 8, 9, 16, 17, 33, 64):
        for tn in (1, 2, 5, 8, 16, 17, 40, 130, 257):
            for g in (1, 2, 4, 8, 16, 32, 64, 128, 256):
                seen = {at(t, tm, tn, g) for t in range(tm * tn)}
                assert seen == {m * 100000 + n for m in range(tm) for n in range(tn)}, (tm, tn, g)
