"""Which kernels the layer operators' calls launch, seen by a stand-in for the HIP runtime (no GPU)."""

import pytest

from tests import hip_stand_in, layer_cases


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return hip_stand_in.built(tmp_path_factory.mktemp("stand_in"))


def test_every_few_row_kernel_is_launched_by_some_call(stand_in):
    got = hip_stand_in.run(stand_in, """
assert lib.layer_create(ctypes.byref(plan), 0) == 0
hip.stand_in_launches()
sizes = [256, 1024, 2048, 4096, 5000, 5008, 8192, 8200, 16384, 16400, 65536, 131072]
seen = {}
for t in (1, 2):
    for m in (1, 4, 5, 8, 9, 16, 17, 32, 33, 48, 64):
        for n in sizes:
            for k in sizes:
                if t == 2 and k % 16: continue
                a = layer.LinearArgs(x=P, w=P, out=P, m=m, n=n, k=k, ldx=k, ldw=k, ldo=n, in_type=t, out_type=1)
                assert call(lib.layer_linear, a) == 0
                for line in hip.stand_in_launches().decode().splitlines():
                    seen.setdefault(line.split()[0], (t, m, n, k))
result = dict(seen=seen, kernels=hip.stand_in_kernels().decode().split())
""")
    kernels = {k for k in got["kernels"] if "ptg_rows_kernel" in k}
    assert kernels and kernels == {k for k in got["seen"] if "ptg_rows_kernel" in k}


def test_every_norm_kernel_is_launched_by_some_call(stand_in):
    got = hip_stand_in.run(stand_in, """
assert lib.layer_create(ctypes.byref(plan), 0) == 0
seen = set()
for n in range(8, 32769, 8):
    for t in (0, 1):
        for o in (0, 1, 2):
            a = layer.RmsnormArgs(x=P, out=P, scale=P if o == 2 else None, m=4, n=n, ldx=n, ldo=n, type=t, out_type=o, eps=1e-6)
            assert lib.layer_rmsnorm(ctypes.byref(a), None) == 0
            if o < 2:
                a = layer.RmsnormGradArgs(dy=P, s=P, dx=P, dweight=P, m=4, n=n, lddy=n, lds=n, lddx=n, type=t, dy_type=o, eps=1e-6)
                assert call(lib.layer_rmsnorm_backward, a) == 0
seen = {line.split()[0] for line in hip.stand_in_launches().decode().splitlines()}
result = dict(seen=sorted(seen), kernels=hip.stand_in_kernels().decode().split())
""")
    kernels = {k for k in got["kernels"] if "ptg_rmsnorm" in k}
    assert kernels and not kernels - set(got["seen"]), sorted(kernels - set(got["seen"]))


WHAT_RUNS = r"""
import re
assert lib.layer_create(ctypes.byref(plan), 0) == 0
hip.stand_in_launches()
def what_runs(kind, m, n, k):
    if kind in ("bf16", "e4m3"):
        a = layer.LinearArgs(x=P, w=P, out=P, m=m, n=n, k=k, ldx=k, ldw=k, ldo=n, in_type=1 + (kind == "e4m3"), out_type=1)
        assert call(lib.layer_linear, a) == 0, (kind, m, n, k)
    else:
        a = layer.LinearGradArgs(dpre=P, x=P, w=P, dx=P if kind == "dx" else None, dw=P if kind == "dw" else None, m=m, n=n, k=k,
                                 lddp=n, ldx=k, ldw=k, lddx=k, lddw=k, dx_type=1, dw_type=0)
        assert call(lib.layer_linear_backward, a) == 0, (kind, m, n, k)
    words = []
    for line in hip.stand_in_launches().decode().splitlines():
        name, gx, gy, block, first, chunks = line.split()
        rows = re.search(r"ptg_rows_kernelILb(\d)ELi(\d)ELi(\d)ELi(\d)", name)
        tiles = re.search(r"ptg_product_kernelILi(\d+)ELi(\d)ELi(\d)", name)
        if rows:
            words.append("rows %s %s %s %s" % (("bf16", "e4m3")[int(rows[1])], rows[2], rows[3], rows[4]) + (" shared" if int(gy) > 1 else ""))
        elif tiles:
            words.append("tiles %s %s %s" % (tiles[1], ("NT", "NN", "TN", "E8")[int(tiles[2])], {"0": "one wave", "2": "dynamic"}[tiles[3]]))
        elif "ptg_product_reduce_kernel" in name:
            words.append("all split" if first == "0" else "last wave split")
        else:
            words.append(name)
    return ", ".join(words)
"""


def test_the_compared_products_are_what_they_say(stand_in):
    cases = layer_cases.LINEAR + layer_cases.BACKWARD
    got = hip_stand_in.run(stand_in, WHAT_RUNS + f"result = [what_runs(*c) for c in {[c[1:] for c in cases]!r}]")
    assert {f"{c[1:]}": g for c, g in zip(cases, got)} == {f"{c[1:]}": c[0] for c in cases}


def test_no_product_of_the_range_runs_otherwise(stand_in):
    """Products over the range that the operators are used in: each runs in a way that the compared ones cover."""
    got = hip_stand_in.run(stand_in, WHAT_RUNS + r"""
import math, random
rng = random.Random(7)
def size(lo, hi, step):
    return max(step, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step)
result = {}
for _ in range(40000):
    kind = rng.choice(["bf16", "e4m3", "dx", "dw"])
    m, n, k = size(1, 16384, 1), size(64, 17000, 8), size(64, 17000, 16 if kind == "e4m3" else 8)
    if rng.random() < 0.5:
        n, k = (n + 63) // 64 * 64, (k + 127) // 128 * 128
    if m * n * k <= 8192 ** 3:
        result.setdefault(what_runs(kind, m, n, k), [kind, m, n, k])
""")
    covered = {c[0] for c in layer_cases.LINEAR + layer_cases.BACKWARD}
    assert len(got) > 40 and not set(got) - covered, {w: got[w] for w in set(got) - covered}
