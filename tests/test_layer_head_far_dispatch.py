"""Which kernels the int8 product, the cross entropy and its gradient launch over all sizes that they take, seen by a stand-in for
the HIP runtime (no GPU)."""

import pytest

from tests import head_cases, head_far_cases, hip_stand_in


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return hip_stand_in.built(tmp_path_factory.mktemp("stand_in"))


@pytest.mark.parametrize("cases", [head_far_cases.CASES, head_far_cases.OUTGROWN], ids=["compared", "outgrown"])
def test_the_calls_are_what_they_say(stand_in, cases):
    got = hip_stand_in.run(stand_in, head_cases.WHAT_RUNS + f"result = [what_runs(*c) for c in {[c[1:] for c in cases]!r}]")
    assert {f"{c[1:]}": g for c, g in zip(cases, got)} == {f"{c[1:]}": c[0] for c in cases}


def test_no_call_of_any_size_runs_otherwise(stand_in):
    """Calls up to the largest vocabulary and the longest rows: each launches what the compared ones cover."""
    got = hip_stand_in.run(stand_in, head_cases.WHAT_RUNS + r"""
import math, random
rng = random.Random(17)
def size(lo, hi, step):
    return max(step, round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step) * step)
result = {}
for _ in range(40000):
    kind = rng.choice(["i8", "i8", "loss", "loss", "dx", "dw"])
    i8 = kind == "i8"
    m = size(1, 64, 1) if rng.random() < 0.5 else size(1, 200000, 1)
    n, k = size(64, 1 << 20, 1 if kind == "loss" else 8), size(64, 131056 if i8 else 1 << 20, 16 if i8 else 8)
    if rng.random() < 0.4:
        n, k = min((n + 63) // 64 * 64, 1 << 20), min((k + 127) // 128 * 128, 130944 if i8 else 1 << 20)
    if n * k <= 1 << 34 and m * k <= 1 << 33 and m * n * k < 1 << 44:
        for part in what_runs(kind, m, n, k).split("; "):
            result.setdefault(part, [kind, m, n, k])
""")
    covered = {part for c in head_cases.CASES + head_far_cases.CASES for part in c[0].split("; ")}
    assert len(got) > 60 and not set(got) - covered, {w: got[w] for w in set(got) - covered}
    assert {c[0].split("; ")[0] for c in head_far_cases.CASES} <= set(got)
