"""Host code of the plans against a stand-in for the HIP runtime: what they wait for, and which streams they touch."""

import pytest

from tests import hip_stand_in


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return hip_stand_in.built(tmp_path_factory.mktemp("stand_in"))


def test_plans_wait_for_the_memory_they_clear(stand_in):
    """A plan's counters are cleared on the null stream. A stream that does not wait for that one (torch's do not) could
    start a kernel before they are."""
    got = hip_stand_in.run(stand_in, """
d = ptg.TileDesc()
assert lib.gemm_default_desc(ctypes.byref(d), 256, 0) == 0
g = ctypes.c_void_p()
status = [lib.gemm_create(ctypes.byref(g), ctypes.byref(d))]
left = [hip.stand_in_unwaited()]
status.append(lib.layer_create(ctypes.byref(plan), 0))
left.append(hip.stand_in_unwaited())
a = layer.LinearArgs(x=P, w=P, out=P, m=1, n=256, k=8192, ldx=8192, ldw=8192, ldo=256, in_type=1, out_type=1)
status.append(call(lib.layer_linear, a, A))
result = dict(status=status, left=left, early=hip.stand_in_early_launches(), launches=hip.stand_in_launches().decode())
""")
    assert got["status"] == [0, 0, 0] and "ptg_rows_kernel" in got["launches"]
    assert got["left"] == [0, 0] and got["early"] == 0
