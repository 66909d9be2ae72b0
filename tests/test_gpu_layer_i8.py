"""The int8 product with its epilogue against the fp64 oracle. Sums of int8 products are exact, so a result is off by the
epilogue's roundings alone: the sum's to fp32, one for each scale and term, and the output's."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests import head_cases
from tests.layer_util import Out, normal, say, within
from tests.test_gpu_layer_linear import LARGE, SHAPES, sampled

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    ptg.layer_sync(p)
    p.destroy()


def codes(seed, m, k, pad=0):
    t = torch.randint(-127, 128, (m, k), generator=torch.Generator().manual_seed(seed), dtype=torch.int8).cuda()
    if not pad:
        return t
    wide = torch.full((m, k + pad), 96, dtype=I8, device="cuda")
    wide[:, :k] = t
    return wide[:, :k]


def scales(seed, n, k=1):
    return (torch.rand(n, generator=torch.Generator().manual_seed(seed)) * 0.02 + 0.001).cuda() / max(k, 1) ** 0.5


def bounds(x, w, bias, act, residual, dtype, xs, ws):
    z, out = ref.linear(x, w, bias, act, residual, xs, ws)
    plain, _ = ref.linear(x, w, None, "none", None, xs, ws)
    err = plain.abs() * 4 * ref.U32 + (0 if bias is None else (z.abs() + ref.d(bias).abs()) * 2 * ref.U32)
    y_err = 1.2 * err + (0 if act in ("none", "relu") else 2.0 ** -18 * z.abs())
    if residual is not None:
        y_err = y_err + (ref.d(residual).abs() + out.abs()) * 2 * ref.U32
    return (z, ref.rounded(z, BF16, err)), (out, ref.rounded(out, dtype, y_err))


def check(plan, m, n, k, out_t=F32, act="none", bias=BF16, residual=BF16, pre=True, pad=0, rows=None):
    x, w, xs, ws = codes(1, m, k, pad), codes(2, n, k, pad), scales(5, m), scales(6, n, k)
    b = None if bias is None else normal(3, n, dtype=bias)
    r = None if residual is None else normal(4, m, n, dtype=residual, pad=pad)
    out, z_out = Out(m, n, out_t), Out(m, n, BF16) if pre else None
    ptg.layer_linear(x, w, out.t, plan, bias=b, activation=act, residual=r, pre=z_out.t if pre else None, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    out.check()
    at = slice(None) if rows is None else rows.cuda()
    z, y = bounds(x[at], w, b, act, None if r is None else r[at], out_t, xs[at], ws)
    within(out.t[at], *y, f"out {m} x {n} x {k}")
    if pre:
        within(z_out.t[at], *z, f"pre {m} x {n} x {k}")
        z_out.check()
    return out.t


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_sizes(plan, m, n, k):
    k = (k + 15) // 16 * 16
    say("int8", m, n, k)
    check(plan, m, n, k, act="gelu")


@pytest.mark.parametrize("m", [1, 20, 150, 520])
@pytest.mark.parametrize("act", ref.ACTIVATIONS)
def test_activations_and_types(plan, m, act):
    say("int8 act", m, act)
    check(plan, m, 264, 528, BF16, act, F32, F32)
    check(plan, m, 264, 528, F32, act, BF16, None, pre=False)


@pytest.mark.parametrize("m", [1, 20, 150, 520])
def test_parts_and_strides(plan, m):
    say("int8 parts", m)
    check(plan, m, 520, 272, bias=None, residual=None, pre=False)
    check(plan, m, 520, 272, BF16, "silu", bias=F32, residual=F32, pre=True, pad=16)
    check(plan, m, 520, 272, bias=None, pre=False, pad=2000)
    check(plan, m, 264, 0, BF16, "silu")


@pytest.mark.parametrize("k", [16, 48, 64, 80, 112, 128, 144, 192, 240, 256, 320, 384, 400, 528, 1040])
@pytest.mark.parametrize("m,n", [(130, 264), (300, 520)])
def test_short_and_odd_k(plan, m, n, k):
    say("int8 short k", m, n, k)
    check(plan, m, n, k)


@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_tiles(plan, m, n, k):
    k = k // 16 * 16
    say("int8 large", m, n, k)
    a = check(plan, m, n, k, BF16, "silu", rows=sampled(m, 256))
    b = check(plan, m, n, k, BF16, "silu", rows=sampled(m, 256)[:1])
    assert torch.equal(a, b), "the same call twice gave different bits"


# w large enough that x goes through LDS: one share of k and several, shares that end inside a segment, a ragged last block of w
@pytest.mark.parametrize("m,n,k", [(8, 8200, 4112), (16, 4104, 8208), (17, 16408, 2064), (24, 2056, 16400), (32, 65544, 528), (32, 4104, 4112),
                                   (33, 8200, 2064), (48, 1032, 32784), (64, 2056, 16400), (64, 33032, 1040), (40, 16392, 1296)])
def test_some_rows_of_a_large_weight(plan, m, n, k):
    say("int8 some rows", m, n, k)
    check(plan, m, n, k, act="silu", pad=48)
    x, w = codes(1, m, k), codes(2, n, k)
    a, b = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    ptg.layer_linear(x, w, a, plan)
    ptg.layer_linear(x, w, b, plan)
    torch.cuda.synchronize()
    assert torch.equal(a, b) and torch.equal(a.cpu(), (x.cpu().float().double() @ w.cpu().float().double().t()).float())


@pytest.mark.parametrize("what,kind,m,n,k", [c for c in head_cases.CASES if c[1] == "i8"])
def test_every_kernel(plan, what, kind, m, n, k):
    say(what, m, n, k)
    check(plan, m, n, k, BF16, "silu", rows=sampled(m, 256)[:200])


@pytest.mark.parametrize("m", [1, 40, 70, 300])
def test_sums_are_exact_to_the_last_bit(plan, m):
    """The largest sums that 32 bits hold, and sums whose low bits fp32 additions would lose on the way."""
    k = 131056
    x, w = torch.full((m, k), -128, dtype=I8, device="cuda"), torch.full((264, k), -128, dtype=I8, device="cuda")
    w[1] = 127
    w[2, ::2] = 127
    w[3, : k // 2] = 127
    w[3, -1] = 1
    out = torch.empty(m, 264, device="cuda")
    ptg.layer_linear(x, w, out, plan)
    torch.cuda.synchronize()
    want = x[:1].cpu().long() @ w.cpu().long().t()
    assert want.max() == 128 * 128 * k and torch.equal(out.cpu(), want.float().expand(m, 264))


@pytest.mark.parametrize("m", [1, 20, 200])
def test_scales_are_optional_and_may_be_anything(plan, m):
    x, w = codes(1, m, 128), codes(2, 264, 128)
    out = torch.empty(m, 264, device="cuda")
    ptg.layer_linear(x, w, out, plan)
    torch.cuda.synchronize()
    assert torch.equal(out.cpu(), (x.cpu().long() @ w.cpu().long().t()).float())
    xs, ws = torch.ones(m, device="cuda"), torch.ones(264, device="cuda")
    xs[0], ws[7] = float("nan"), 0.0
    ptg.layer_linear(x, w, out, plan, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    assert torch.isnan(out[0]).all() and (out[1:, 7] == 0).all() and torch.isfinite(out[1:]).all()


@pytest.mark.parametrize("m", [1, 40, 300])
def test_residual_in_place(plan, m):
    x, w, r = codes(1, m, 272), codes(2, 520, 272), normal(4, m, 520)
    fresh = torch.empty_like(r)
    ptg.layer_linear(x, w, fresh, plan, residual=r, x_scale=scales(5, m))
    ptg.layer_linear(x, w, r, plan, residual=r, x_scale=scales(5, m))
    torch.cuda.synchronize()
    assert torch.equal(fresh, r)


def test_refusals(plan):
    x, w, out = codes(1, 4, 64), codes(2, 32, 64), torch.empty(4, 32, dtype=BF16, device="cuda")
    for args in ((x, w.to(BF16), out), (x.to(BF16), w, out), (x.to(torch.uint8), w.to(torch.uint8), out), (x, w, out.to(I8)),
                 (x, codes(2, 32, 80), out)):
        with pytest.raises(ValueError):
            ptg.layer_linear(*args, plan)
    for k in (72, 131072):
        with pytest.raises(ptg.PtgError) as e:
            ptg.layer_linear(codes(1, 4, k), codes(2, 32, k), out, plan)
        assert e.value.status == -2
    with pytest.raises(ValueError):
        ptg.layer_linear_backward(out, x, None, plan, dw=torch.empty(32, 64, device="cuda"))
