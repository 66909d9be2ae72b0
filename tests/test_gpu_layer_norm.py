"""The RMS norm with the residual's addition and its gradient against the fp64 oracle."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import Out, normal, say, within

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
EPS = 1e-6


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    p.destroy()


def check_norm(m, n, t, out_t, residual, weight_t=BF16, pad=0, eps=EPS, x=None):
    x = normal(1, m, n, scale=3.0, dtype=t, pad=pad) if x is None else x
    res = normal(2, m, n, dtype=t, pad=pad) if residual else None
    w = None if weight_t is None else (1 + 0.2 * normal(3, n, dtype=F32)).to(weight_t)
    out, s_out = Out(m, n, out_t), Out(m, n, t)
    scale = torch.full((m,), -1.0, device="cuda") if out_t == E4M3 else None
    ptg.layer_rmsnorm(x, w, out.t, residual=res, sum_out=s_out.t, scale=scale, eps=eps)
    torch.cuda.synchronize()
    s, y = ref.rmsnorm(x, w, res, eps)
    within(s_out.t, s, ref.rounded(s, t, s.abs() * 2 * ref.U32), "sum")
    if out_t == E4M3:
        want, v = ref.quantise(y)
        within(scale, want, want * 100 * ref.U32, "scale")
        within(out.t.float(), v, ref.rmsnorm_bound(v, E4M3, n), "codes")
        if m:
            assert ((out.t.float().abs().amax(dim=1) == 448) | (scale == 1)).all()
    else:
        within(out.t, y, ref.rmsnorm_bound(y, out_t, n), "out")
    out.check()
    s_out.check()


# row-group sizes change at n = 2048 and 8192, chunks per thread in between; ragged n everywhere
SIZES = [(1, 8), (3, 64), (5, 512), (7, 520), (4, 2048), (9, 2056), (2, 4096), (3, 5000), (1, 8192), (6, 8200), (2, 16384), (2, 32768)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("out_t", [BF16, F32, E4M3])
@pytest.mark.parametrize("t", [BF16, F32])
def test_norm_sizes(m, n, t, out_t):
    say("norm", m, n, t, out_t)
    check_norm(m, n, t, out_t, True)


@pytest.mark.parametrize("out_t", [BF16, E4M3])
def test_norm_variants(out_t):
    say("norm variants", out_t)
    check_norm(33, 776, BF16, out_t, False)
    check_norm(33, 776, BF16, out_t, True, weight_t=None)
    check_norm(33, 776, F32, out_t, True, weight_t=F32, pad=24)
    check_norm(600, 1024, BF16, out_t, True, pad=8)
    check_norm(1, 776, BF16, out_t, True, eps=0.5)


def test_norm_in_place_and_without_sum():
    m, n = 37, 3000
    x, r = normal(1, m, n), normal(2, m, n)
    s, y = ref.rmsnorm(x, None, r)
    for target in ("x", "residual"):
        a, b = x.clone(), r.clone()
        out = torch.empty_like(x)
        ptg.layer_rmsnorm(a, None, out, residual=b, sum_out=a if target == "x" else b)
        torch.cuda.synchronize()
        within(a if target == "x" else b, s, ref.rounded(s, BF16, s.abs() * 2 * ref.U32), "sum " + target)
        within(out, y, ref.rmsnorm_bound(y, BF16, n), "out " + target)
        assert torch.equal(b if target == "x" else a, r if target == "x" else x)
    out = torch.empty_like(x)
    ptg.layer_rmsnorm(x, None, out, residual=r)
    torch.cuda.synchronize()
    within(out, y, ref.rmsnorm_bound(y, BF16, n), "no sum")


@pytest.mark.parametrize("n", [264, 4104, 9000])
def test_norm_zero_small_and_non_finite_rows(n):
    say("norm special rows", n)
    x = normal(4, 8, n, dtype=F32)
    x[1] = 0.0
    x[2] = 1e-30           # eps decides: y = 1e-27
    x[3, n // 2] = float("nan")
    x[4, n - 1] = float("inf")
    x[5] = 1e-39           # y / 448 falls below 2^-126: the scale stops there
    x[6] *= 1e15
    good = [0, 1, 2, 5, 6, 7]
    out, scale = torch.zeros(8, n, dtype=E4M3, device="cuda"), torch.zeros(8, device="cuda")
    full = torch.zeros(8, n, device="cuda")
    ptg.layer_rmsnorm(x, None, out, scale=scale)
    ptg.layer_rmsnorm(x, None, full)
    torch.cuda.synchronize()
    assert torch.isnan(scale[3:5]).all() and torch.isnan(out.float()[3:5]).all()
    assert torch.isnan(full[3]).all() and torch.isnan(full[4, n - 1]) and (full[4, : n - 1] == 0).all()
    _, y = ref.rmsnorm(x[good], None)
    want, v = ref.quantise(y)
    within(full[good], y, ref.rmsnorm_bound(y, F32, n), "full")
    within(scale[good], want, want * 100 * ref.U32, "scale")
    within(out.float()[good], v, ref.rmsnorm_bound(v, E4M3, n), "codes")
    assert scale[1] == 1 and (out.float()[1] == 0).all()
    # a NaN in the weight reaches every row's scale
    w = torch.ones(n, device="cuda")
    w[5] = float("nan")
    ptg.layer_rmsnorm(x[:1].contiguous(), w, out[:1], scale=scale[:1])
    torch.cuda.synchronize()
    assert torch.isnan(scale[0]) and torch.isnan(out.float()[0]).all()


def test_norm_of_no_rows_writes_nothing():
    out = Out(0, 64, BF16)
    ptg.layer_rmsnorm(normal(1, 0, 64), None, out.t)
    torch.cuda.synchronize()
    out.check()


def check_backward(plan, m, n, t, dy_t, dsum, weight_t=BF16, pad=0, eps=EPS):
    s, dy = normal(1, m, n, scale=2.0, dtype=t, pad=pad), normal(2, m, n, dtype=dy_t, pad=pad)
    w = None if weight_t is None else (1 + 0.2 * normal(3, n, dtype=F32)).to(weight_t)
    ds = normal(4, m, n, dtype=t, pad=pad) if dsum else None
    dx, dw = Out(m, n, t), torch.full((n + 8,), -7.0, device="cuda")
    ptg.layer_rmsnorm_backward(dy, s, w, dx.t, dw[:n], plan, dsum=ds, eps=eps)
    torch.cuda.synchronize()
    want_dx, want_dw = ref.rmsnorm_backward(dy, s, w, ds, eps)
    b_dx, b_dw = ref.rmsnorm_backward_bounds(dy, s, w, ds, t, eps)
    within(dx.t, want_dx, b_dx, "dx")
    within(dw[:n], want_dw, b_dw, "dweight")
    dx.check()
    assert (dw[n:] == -7.0).all()


@pytest.mark.parametrize("m,n", SIZES + [(1111, 264), (2100, 2048), (700, 4104), (300, 16384)])
@pytest.mark.parametrize("t,dy_t", [(BF16, BF16), (F32, BF16), (BF16, F32)])
def test_norm_backward_sizes(plan, m, n, t, dy_t):
    say("norm backward", m, n, t, dy_t)
    check_backward(plan, m, n, t, dy_t, True)


def test_norm_backward_variants(plan):
    say("norm backward variants")
    check_backward(plan, 50, 1000, BF16, BF16, False)
    check_backward(plan, 50, 1000, F32, F32, False, weight_t=None)
    check_backward(plan, 50, 1000, F32, F32, True, weight_t=F32, pad=40)
    check_backward(plan, 50, 3000, BF16, BF16, True, eps=0.3)


def test_norm_backward_parts_accumulate_and_alias(plan):
    m, n = 77, 1032
    s, dy, w, ds = normal(1, m, n), normal(2, m, n), normal(3, n), normal(4, m, n)
    want_dx, want_dw = ref.rmsnorm_backward(dy, s, w, ds)
    b_dx, b_dw = ref.rmsnorm_backward_bounds(dy, s, w, ds, BF16)
    both_dx, both_dw = torch.empty_like(s), torch.empty(n, device="cuda")
    ptg.layer_rmsnorm_backward(dy, s, w, both_dx, both_dw, plan, dsum=ds)
    only_dx, only_dw = torch.empty_like(s), torch.empty(n, device="cuda")
    ptg.layer_rmsnorm_backward(dy, s, w, only_dx, None, plan, dsum=ds)
    ptg.layer_rmsnorm_backward(dy, s, w, None, only_dw, plan, dsum=ds)
    ptg.layer_rmsnorm_backward(dy, s, w, ds, None, plan, dsum=ds)  # dx in place of dsum
    torch.cuda.synchronize()
    within(both_dx, want_dx, b_dx, "dx")
    within(both_dw, want_dw, b_dw, "dweight")
    assert torch.equal(only_dx, both_dx) and torch.equal(only_dw, both_dw) and torch.equal(ds, both_dx)
    acc = torch.full((n,), 3.0, device="cuda")
    ptg.layer_rmsnorm_backward(dy, s, w, None, acc, plan, accumulate=True)
    torch.cuda.synchronize()
    within(acc, want_dw + 3.0, b_dw + 32 * ref.U32, "accumulated")
    # no rows: a zero gradient, or nothing added
    e = torch.empty(0, n, dtype=BF16, device="cuda")
    ptg.layer_rmsnorm_backward(e, e, w, None, acc, plan, accumulate=True)
    torch.cuda.synchronize()
    assert (acc != 0).any()
    ptg.layer_rmsnorm_backward(e, e, w, e, acc, plan)
    torch.cuda.synchronize()
    assert (acc == 0).all()


def test_norm_gradient_against_differences(plan):
    m, n = 6, 264
    s, dy, w = normal(1, m, n, dtype=F32), normal(2, m, n, dtype=F32), normal(3, n, dtype=F32)
    dx, dw = torch.empty_like(s), torch.empty_like(w)
    ptg.layer_rmsnorm_backward(dy, s, w, dx, dw, plan)
    torch.cuda.synchronize()
    h = 1e-5
    for seed in range(3):
        u, v = ref.d(normal(30 + seed, m, n, dtype=F32)), ref.d(normal(40 + seed, n, dtype=F32))
        loss = lambda t: (ref.rmsnorm(ref.d(s) + t * u, ref.d(w) + t * v)[1] * ref.d(dy)).sum()  # noqa: E731
        diff = (loss(h) - loss(-h)) / (2 * h)
        got = (ref.d(dx) * u).sum() + (ref.d(dw) * v).sum()
        size = (ref.d(dx) * u).abs().sum() + (ref.d(dw) * v).abs().sum()
        assert abs(diff - got) <= size * 1e-5
