"""Rows enough that every row group of the norms, and every wave of the activation's gradient, goes through its loop more
than twice: the next row's loads, the two LDS buffers in turn, sums that stay in registers. (256 CUs: the forward norm has
4096, 1024 or 256 groups, changing at n = 1024 and 4096, its gradient 2048, 512 or 256.) m is a multiple of no group count."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import Out, normal, say, within
from tests.test_gpu_layer_norm import check_backward, check_norm

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn

# one and two chunks a thread of 64, 256 and 1024 threads, and four of 1024, the last one ragged
FORWARD = [(9000, 264), (9000, 776), (2500, 1032), (2500, 2056), (700, 8200), (700, 12296), (600, 24584)]
BACKWARD = [(5000, 264), (5000, 776), (1300, 2000), (1300, 2056), (700, 8200), (700, 12296), (600, 24584)]


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    p.destroy()


@pytest.mark.parametrize("m,n", FORWARD)
@pytest.mark.parametrize("t,out_t", [(BF16, BF16), (BF16, E4M3), (F32, F32), (F32, E4M3)])
def test_norm(m, n, t, out_t):
    say("norm", m, n, t, out_t)
    check_norm(m, n, t, out_t, True, pad=8)


@pytest.mark.parametrize("m,n", FORWARD)
def test_norm_with_the_sum_in_place(m, n):
    say("norm in place", m, n)
    x, r = normal(1, m, n), normal(2, m, n)
    s, y = ref.rmsnorm(x, None, r)
    out = torch.empty_like(x)
    ptg.layer_rmsnorm(x, None, out, residual=r, sum_out=r)
    torch.cuda.synchronize()
    within(r, s, ref.rounded(s, BF16, s.abs() * 2 * ref.U32), "sum")
    within(out, y, ref.rmsnorm_bound(y, BF16, n), "out")


@pytest.mark.parametrize("m,n", BACKWARD)
@pytest.mark.parametrize("t,dy_t", [(BF16, BF16), (F32, BF16), (F32, F32)])
def test_norm_backward(plan, m, n, t, dy_t):
    say("norm backward", m, n, t, dy_t)
    check_backward(plan, m, n, t, dy_t, True, pad=8)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("m,n", [(5000, 8200), (40001, 520), (3000, 16392)])  # 42, 40 and 48 rows a workgroup of four waves
def test_activation_backward(plan, m, n, act):
    say("activation backward", m, n, act)
    do, z = normal(1, m, n, pad=8), normal(2, m, n, scale=2.0, pad=16)
    dpre, db = Out(m, n, BF16), torch.full((n + 8,), -7.0, device="cuda")
    ptg.layer_activation_backward(do, None if act == "none" else z, dpre.t, plan, activation=act, dbias=db[:n])
    torch.cuda.synchronize()
    g = torch.ones_like(ref.d(z)) if act == "none" else ref.act_grad(ref.d(z), act)
    bp, bb = ref.activation_backward_bounds(do, z, act)
    within(dpre.t, ref.d(do) * g, bp, "dpre")
    within(db[:n], (ref.d(do) * g).sum(dim=0), bb, "dbias")
    dpre.check()
    assert (db[n:] == -7.0).all()
