"""Which kernels the layer operators' calls launch, seen by a stand-in for the HIP runtime (no GPU)."""

import pytest

from tests import hip_stand_in


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
