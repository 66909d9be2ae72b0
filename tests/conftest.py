import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running CPU test")


def pytest_collection_modifyitems(items):
    """Tests that need two streams to run side by side go first: streams share four hardware queues, dealt out as streams come
    into use, so the more of them other tests have used, the sooner two of these tests' own meet on one queue and run in turn."""
    items.sort(key=lambda item: "partial_occupancy" not in item.name)


@pytest.fixture(scope="session")
def repo_root():
    return ROOT
