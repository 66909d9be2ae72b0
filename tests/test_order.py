"""The order that the suite runs in."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_tests_that_need_streams_side_by_side_go_first():
    out = subprocess.run([sys.executable, "-m", "pytest", "tests", "--collect-only", "-q", "-m", "gpu", "-p", "no:cacheprovider"], cwd=ROOT,
                         capture_output=True, text=True, check=True).stdout
    names = [x for x in out.splitlines() if "::" in x]
    first = [x for x in names if "partial_occupancy" in x]
    assert len(first) >= 2 and names[: len(first)] == first
