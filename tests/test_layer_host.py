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


# a product in 256 x 256 tiles on stream A, then a call that runs no such tiles on stream B
TWO_STREAMS = """
assert lib.layer_create(ctypes.byref(plan), 0) == 0
product = layer.LinearArgs(x=P, w=P, out=P, m=8192, n=8192, k=8192, ldx=8192, ldw=8192, ldo=8192, in_type=1, out_type=1)
norm = layer.RmsnormGradArgs(dy=P, s=P, dx=P, dweight=P, m=64, n=512, lddy=512, lds=512, lddx=512, type=1, dy_type=1, eps=1e-6)
status = [call(lib.layer_linear, product, A), call(lib.layer_rmsnorm_backward, norm, B)]
launches = hip.stand_in_launches().decode()
hip.stand_in_end_stream(A)
"""


def test_a_stream_may_end_after_the_plans_next_call(stand_in):
    got = hip_stand_in.run(stand_in, TWO_STREAMS + """
status += [lib.layer_sync(plan), lib.layer_destroy(plan)]
result = dict(status=status, dead=hip.stand_in_dead_uses(), launches=launches)
""")
    assert "ptg_product_kernelILi256" in got["launches"] and "ptg_rmsnorm_backward" in got["launches"]
    assert got["status"] == [0, 0, 0, 0] and got["dead"] == 0


def test_layer_sync_reports_the_status_of_products_on_earlier_streams(stand_in):
    got = hip_stand_in.run(stand_in, TWO_STREAMS + """
hip.stand_in_device_status(1)
status += [lib.layer_sync(plan), lib.layer_sync(plan), lib.layer_destroy(plan)]
result = dict(status=status, dead=hip.stand_in_dead_uses())
""")
    assert got["status"] == [0, 0, -7, 0, 0] and got["dead"] == 0  # GEMM_E_TIMEOUT once, then cleared


# the plain plan's run or the layer plan's call on stream A, and its synchronisation
SYNCED = """
d, g = ptg.TileDesc(), ctypes.c_void_p()
assert lib.gemm_default_desc(ctypes.byref(d), 256, 0) == 0 and lib.gemm_create(ctypes.byref(g), ctypes.byref(d)) == 0
assert lib.layer_create(ctypes.byref(plan), 0) == 0
lib.gemm_run.argtypes = [ctypes.c_void_p] * 3 + [ctypes.c_int64] * 3 + [ctypes.c_int32] + [ctypes.c_void_p] * 2
norm = layer.RmsnormGradArgs(dy=P, s=P, dx=P, m=64, n=512, lddy=512, lds=512, lddx=512, type=1, dy_type=1, eps=1e-6)
def run(s):
    return lib.gemm_run(P, P, P, 512, 512, 512, 2, g, s), call(lib.layer_rmsnorm_backward, norm, s)
hip.stand_in_capture({captured})
status = [*run(A), lib.gemm_sync(g), lib.layer_sync(plan)]
hip.stand_in_capture(0)
"""


def test_a_stream_may_end_after_a_sync(stand_in):
    got = hip_stand_in.run(stand_in, SYNCED.format(captured=0) + """
hip.stand_in_end_stream(A)
status += [lib.gemm_sync(g), lib.layer_sync(plan), *run(B), *run(A.__class__(0x3000))]
dead = hip.stand_in_dead_uses()
status += [lib.gemm_destroy(g), lib.layer_destroy(plan)]
result = dict(status=status, dead=[dead, hip.stand_in_dead_uses()])
""")
    assert got["status"] == [0] * 12 and got["dead"] == [0, 0]


def test_a_captured_stream_is_kept(stand_in):
    """Replays may be under way on it after a sync: a run on another stream still waits for them."""
    got = hip_stand_in.run(stand_in, SYNCED.format(captured=1) + """
before = hip.stand_in_waits()
status += [*run(B)]
result = dict(status=status, waits=hip.stand_in_waits() - before)
""")
    assert got["status"] == [0] * 6 and got["waits"] == 2


def test_the_e4m3_probe_refuses(stand_in):
    got = hip_stand_in.run(stand_in, """
c, out = bytes(256), ctypes.c_float()
def f(device, form, a, b, n):
    return lib.gemm_e4m3_probe(device, form, a, b, n, ctypes.byref(out))
result = [f(0, 4, c, c, 1), f(0, -1, c, c, 1), f(0, 0, None, c, 1), f(0, 0, c, None, 1), f(0, 0, c, c, -1), f(1, 0, c, c, 1)] + \\
    [f(0, form, c, c, n) for form, n in ((0, 33), (1, 17), (2, 129), (3, 65))] + [f(0, 2, c, c, 128)]
""")
    assert got == [-1, -1, -1, -1, -1, -4, -1, -1, -1, -1, 0]
