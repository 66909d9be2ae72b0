"""The product with bias, activation and residual in its epilogue, and its gradients, against the fp64 oracle."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import Out, normal, say, within

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    ptg.layer_sync(p)
    p.destroy()


@pytest.fixture(scope="module")
def streams():
    """The two streams beside the default one that all tests here share (streams share few hardware queues: tests that
    count on work under way at once fare better with fewer of them in a process)."""
    return torch.cuda.Stream(), torch.cuda.Stream()


def operands(m, n, k, t, pad=0):
    if t == E4M3:
        x, w = normal(1, m, k, scale=60.0, dtype=E4M3, pad=pad), normal(2, n, k, scale=60.0, dtype=E4M3, pad=pad)
        xs = torch.rand(m, generator=torch.Generator().manual_seed(5)).cuda() * 0.02 + 0.001
        ws = (torch.rand(n, generator=torch.Generator().manual_seed(6)).cuda() * 0.02 + 0.001) / max(k, 1) ** 0.5
        return x, w, xs, ws
    return normal(1, m, k, pad=pad), normal(2, n, k, scale=max(k, 1) ** -0.5, pad=pad), None, None


def check_linear(plan, m, n, k, t=BF16, out_t=BF16, act="none", bias=BF16, residual=BF16, pre=True, pad=0):
    x, w, xs, ws = operands(m, n, k, t, pad)
    b = None if bias is None else normal(3, n, dtype=bias)
    r = None if residual is None else normal(4, m, n, dtype=residual, pad=pad)
    out, z_out = Out(m, n, out_t), Out(m, n, BF16) if pre else None
    ptg.layer_linear(x, w, out.t, plan, bias=b, activation=act, residual=r, pre=z_out.t if pre else None, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    z, y = ref.linear(x, w, b, act, r, xs, ws)
    bz, by = ref.linear_bounds(x, w, b, act, r, out_t, xs, ws)
    within(out.t, y, by, f"out {m} x {n} x {k}")
    out.check()
    if pre:
        within(z_out.t, z, bz, f"pre {m} x {n} x {k}")
        z_out.check()


# rows from a decode step to several tiles; edges inside a tile, a k-step and a fragment
SHAPES = [(1, 8, 8), (1, 264, 2056), (2, 1000, 520), (3, 8192, 64), (5, 40, 8200), (16, 776, 1032), (17, 520, 264), (24, 64, 16400),
          (33, 1024, 512), (48, 264, 1000), (64, 256, 4104), (65, 512, 256), (100, 136, 776), (128, 128, 96), (129, 264, 40),
          (255, 256, 32), (256, 512, 520), (257, 520, 264), (300, 1000, 72), (777, 520, 136)]


@pytest.mark.parametrize("m,n,k", SHAPES)
@pytest.mark.parametrize("t", [BF16, E4M3])
def test_linear_sizes(plan, m, n, k, t):
    if t == E4M3:
        k = (k + 15) // 16 * 16
    say("linear", m, n, k, t)
    check_linear(plan, m, n, k, t, act="gelu", out_t=BF16)


@pytest.mark.parametrize("m", [1, 20, 150, 520])
@pytest.mark.parametrize("act", ref.ACTIVATIONS)
def test_linear_activations_and_types(plan, m, act):
    say("linear act", m, act)
    check_linear(plan, m, 264, 528, BF16, F32, act, BF16, F32)
    check_linear(plan, m, 264, 528, E4M3, F32, act, F32, None, pre=False)


@pytest.mark.parametrize("m", [1, 20, 150, 520])
def test_linear_parts(plan, m):
    say("linear parts", m)
    check_linear(plan, m, 520, 264, bias=None, residual=None, pre=False)
    check_linear(plan, m, 520, 264, bias=F32, residual=None, pre=True, pad=8)
    check_linear(plan, m, 520, 272, E4M3, bias=None, residual=BF16, pre=True, pad=16)
    check_linear(plan, m, 520, 272, E4M3, F32, "silu", bias=BF16, residual=F32, pre=False, pad=48)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_linear_empty_sums(plan, m):
    say("linear k = 0", m)
    check_linear(plan, m, 264, 0, act="silu")


def test_linear_of_nothing_writes_nothing(plan):
    out = Out(0, 64, BF16)
    ptg.layer_linear(normal(1, 0, 32), normal(2, 64, 32), out.t, plan)
    ptg.layer_linear(normal(1, 4, 32), normal(2, 0, 32), torch.empty(4, 0, dtype=BF16, device="cuda"), plan)
    torch.cuda.synchronize()
    out.check()


@pytest.mark.parametrize("m", [1, 40, 300])
@pytest.mark.parametrize("t", [BF16, F32])
def test_linear_residual_in_place(plan, m, t):
    x, w, _, _ = operands(m, 520, 264, BF16)
    r = normal(4, m, 520, dtype=t)
    fresh = torch.empty_like(r)
    ptg.layer_linear(x, w, fresh, plan, residual=r)
    ptg.layer_linear(x, w, r, plan, residual=r)
    torch.cuda.synchronize()
    assert torch.equal(fresh, r)


@pytest.mark.parametrize("m", [1, 20, 200])
@pytest.mark.parametrize("t", [BF16, E4M3])
def test_linear_scales_are_optional(plan, m, t):
    x, w = normal(1, m, 128, dtype=t), normal(2, 264, 128, dtype=t)
    out = torch.empty(m, 264, device="cuda")
    ptg.layer_linear(x, w, out, plan)
    torch.cuda.synchronize()
    within(out, ref.d(x) @ ref.d(w).t(), ref.linear_bounds(x, w, None, "none", None, F32)[1], "no scales")


@pytest.mark.parametrize("m", [2, 200])
def test_linear_non_finite(plan, m):
    """An infinity or NaN in one row of x stays in that row, one in a row of w in that column; activations of
    infinite arguments are their limits."""
    x, w, _, _ = operands(m, 264, 128, BF16)
    x[1, 5] = float("nan")
    w[7] = 0.0
    for act, at_minus in (("none", -float("inf")), ("relu", 0.0), ("gelu", 0.0), ("gelu_tanh", 0.0), ("silu", 0.0)):
        out = torch.empty(m, 264, device="cuda")
        b = torch.zeros(264, device="cuda")
        b[3], b[4] = float("inf"), -float("inf")
        ptg.layer_linear(x, w, out, plan, bias=b, activation=act)
        torch.cuda.synchronize()
        assert torch.isnan(out[1]).all(), act
        ok = torch.cat([out[:1], out[2:]])
        assert (ok[:, 3] == float("inf")).all() and (ok[:, 4] == at_minus).all(), act
        assert torch.isfinite(ok[:, 5:]).all() and (ok[:, 7] == 0).all(), act


@pytest.mark.parametrize("act", ref.ACTIVATIONS)
@pytest.mark.parametrize("m,n", [(1, 8), (1, 2056), (7, 520), (64, 512), (130, 1032), (1000, 264), (333, 4104), (70, 16384)])
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


def test_activation_backward_extremes_parts_and_accumulation(plan):
    z = torch.tensor([[-float("inf"), -1e30, -100.0, -0.0, 0.0, 100.0, 1e30, float("inf")]] * 3).to(BF16).cuda()
    do = torch.full((3, 8), 2.0, dtype=BF16, device="cuda")
    for act in ref.ACTIVATIONS[1:]:
        dpre, db = torch.empty_like(do), torch.full((8,), 1.0, device="cuda")
        ptg.layer_activation_backward(do, z, dpre, plan, activation=act, dbias=db, accumulate=True)
        torch.cuda.synchronize()
        mid = 0.0 if act == "relu" else 1.0
        want = torch.tensor([0.0, 0.0, 0.0, mid, mid, 2.0, 2.0, 2.0])
        assert (dpre.float().cpu() - want).abs().max() < 1e-6, act
        assert (db.cpu() - (1 + 3 * want)).abs().max() < 1e-5, act
    a, z = normal(1, 60, 264), normal(2, 60, 264)
    whole, db = torch.empty_like(a), torch.empty(264, device="cuda")
    ptg.layer_activation_backward(a, z, whole, plan, activation="silu", dbias=db)
    only, in_place, over_pre = torch.empty(264, device="cuda"), a.clone(), z.clone()
    ptg.layer_activation_backward(a, z, None, plan, activation="silu", dbias=only)
    ptg.layer_activation_backward(in_place, z, in_place, plan, activation="silu")
    ptg.layer_activation_backward(a, over_pre, over_pre, plan, activation="silu")
    torch.cuda.synchronize()
    assert torch.equal(db, only) and torch.equal(whole, in_place) and torch.equal(whole, over_pre)
    e = torch.empty(0, 264, dtype=BF16, device="cuda")
    ptg.layer_activation_backward(e, e, e, plan, activation="silu", dbias=only, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(db, only)
    ptg.layer_activation_backward(e, e, e, plan, activation="silu", dbias=only)
    torch.cuda.synchronize()
    assert (only == 0).all()


def check_backward(plan, m, n, k, dx_t=BF16, dw_t=F32, accumulate=False, pad=0):
    dpre, x = normal(1, m, n, scale=0.1, pad=pad), normal(2, m, k, pad=pad)
    w = normal(3, n, k, scale=k ** -0.5, pad=pad)
    old = normal(4, n, k, dtype=dw_t) if accumulate else None
    dx, dw = Out(m, k, dx_t), Out(n, k, dw_t, fill=old)
    ptg.layer_linear_backward(dpre, x, w, plan, dx=dx.t, dw=dw.t, accumulate=accumulate)
    torch.cuda.synchronize()
    within(dx.t, *ref.product_bound(dpre, w, dx_t), f"dx {m} {n} {k}")
    within(dw.t, *ref.product_bound(dpre.t(), x, dw_t, old), f"dw {m} {n} {k}")
    dx.check()
    dw.check()


@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (1, 264, 520), (3, 1000, 64), (16, 520, 264), (31, 40, 776), (33, 256, 256), (64, 776, 136),
                                   (100, 264, 1032), (255, 520, 40), (257, 264, 264), (777, 136, 520), (1025, 520, 264)])
def test_linear_backward_sizes(plan, m, n, k):
    say("linear backward", m, n, k)
    check_backward(plan, m, n, k)


def test_linear_backward_variants(plan):
    say("linear backward variants")
    check_backward(plan, 70, 264, 520, F32, BF16)
    check_backward(plan, 70, 264, 520, accumulate=True, pad=24)
    check_backward(plan, 300, 264, 520, F32, BF16, accumulate=True, pad=8)
    dpre, x, w = normal(1, 70, 264), normal(2, 70, 520), normal(3, 264, 520)
    dx, dw = torch.empty(70, 520, dtype=BF16, device="cuda"), torch.empty(264, 520, device="cuda")
    ptg.layer_linear_backward(dpre, x, w, plan, dx=dx, dw=dw)
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    ptg.layer_linear_backward(dpre, None, w, plan, dx=dx2)
    ptg.layer_linear_backward(dpre, x, None, plan, dw=dw2)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    e = torch.empty(0, 264, dtype=BF16, device="cuda")
    ptg.layer_linear_backward(e, torch.empty(0, 520, dtype=BF16, device="cuda"), None, plan, dw=dw2, accumulate=True)
    torch.cuda.synchronize()
    assert torch.equal(dw, dw2)
    ptg.layer_linear_backward(e, torch.empty(0, 520, dtype=BF16, device="cuda"), None, plan, dw=dw2)
    torch.cuda.synchronize()
    assert (dw2 == 0).all()


def test_layer_gradient_against_differences(plan):
    """out = act(x w^T + b): the three gradients along random directions against central differences. The chain
    rounds dpre to bf16 (half a step: 2^-8 of each product's terms) and dx once more."""
    m, n, k = 24, 136, 264
    x, w, b, do = normal(1, m, k), normal(2, n, k, scale=k ** -0.5), normal(3, n), normal(4, m, n)
    out, pre, dpre = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(3))
    dx, dw, db = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    for act in ref.ACTIVATIONS:
        if act == "relu":
            continue  # not differentiable where a difference may cross it
        ptg.layer_linear(x, w, out, plan, bias=b, activation=act, pre=pre)
        ptg.layer_activation_backward(do, pre, dpre, plan, activation=act, dbias=db)
        ptg.layer_linear_backward(dpre, x, w, plan, dx=dx, dw=dw)
        torch.cuda.synchronize()
        u, v, q = ref.d(normal(5, m, k, dtype=F32)), ref.d(normal(6, n, k, dtype=F32)), ref.d(normal(7, n, dtype=F32))
        h = 1e-5
        loss = lambda t: (ref.linear(ref.d(x) + t * u, ref.d(w) + t * v, ref.d(b) + t * q, act)[1] * ref.d(do)).sum()  # noqa: E731
        diff = (loss(h) - loss(-h)) / (2 * h)
        got = (ref.d(dx) * u).sum() + (ref.d(dw) * v).sum() + (ref.d(db) * q).sum()
        # every term of the directional derivative, in magnitude; pre's rounding moves act' by at most |z| 2^-8
        # times its slope (at most 1), dpre's rounding by 2^-8 of itself
        dir_z = (u.abs() @ ref.d(w).abs().t()) + (ref.d(x).abs() @ v.abs().t()) + q.abs()
        z = ref.linear(x, w, b)[0]
        size = (ref.d(do).abs() * dir_z * (z.abs() * 2.0 ** -8 + 1.2 * 2.0 ** -8)).sum()
        assert abs(diff - got) <= size, (act, float(diff), float(got), float(size))


def test_calls_on_two_streams_are_ordered(plan, streams):
    """One plan, two streams without a wait between them: the plan's scratch serves one call at a time."""
    m, n, k = 200, 520, 264
    x, w = normal(1, m, k), normal(2, n, k)
    dpre, pre = normal(3, m, n), normal(4, m, n)
    want, dw_want, db_want = torch.empty(m, n, device="cuda"), torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda")
    ptg.layer_linear(x, w, want, plan)
    ptg.layer_linear_backward(dpre, x, None, plan, dw=dw_want)
    ptg.layer_activation_backward(dpre, pre, None, plan, activation="silu", dbias=db_want)
    torch.cuda.synchronize()
    a, b = streams
    outs = []
    for i in range(6):
        s = a if i % 2 else b
        o, dw, db = torch.empty_like(want), torch.empty_like(dw_want), torch.empty_like(db_want)
        s.wait_stream(torch.cuda.current_stream())
        ptg.layer_linear(x, w, o, plan, stream=s)
        ptg.layer_linear_backward(dpre, x, None, plan, dw=dw, stream=s)
        ptg.layer_activation_backward(dpre, pre, None, plan, activation="silu", dbias=db, stream=s)
        outs.append((o, dw, db))
    torch.cuda.synchronize()
    for o, dw, db in outs:
        assert torch.equal(o, want) and torch.equal(dw, dw_want) and torch.equal(db, db_want)
    ptg.layer_sync(plan)


@pytest.mark.parametrize("m", [1, 40, 300])
def test_layer_step_replays_from_a_graph(plan, streams, m):
    """Forward and backward calls captured once and replayed over changing inputs, with the plan's own uncaptured calls
    between the replays."""
    n, k = 520, 264
    x, w, b, do, g = normal(1, m, k), normal(2, n, k, scale=0.06), normal(3, n), normal(4, m, n), normal(5, k)
    y = torch.empty_like(x)
    out, pre, dpre = (torch.empty(m, n, dtype=BF16, device="cuda") for _ in range(3))
    dy, dxn = torch.empty_like(x), torch.empty_like(x)
    dw, db, dg = torch.empty(n, k, device="cuda"), torch.empty(n, device="cuda"), torch.empty(k, device="cuda")

    def step():
        ptg.layer_rmsnorm(x, g, y)
        ptg.layer_linear(y, w, out, plan, bias=b, activation="gelu", pre=pre)
        ptg.layer_activation_backward(do, pre, dpre, plan, activation="gelu", dbias=db)
        ptg.layer_linear_backward(dpre, y, w, plan, dx=dy, dw=dw)
        ptg.layer_rmsnorm_backward(dy, x, g, dxn, dg, plan)

    results = (out, pre, dpre, dy, dxn, dw, db, dg)
    s = streams[0]
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for i in range(4):
            x.copy_(normal(50 + i, m, k))
            step()
            s.synchronize()
            want = [t.clone() for t in results]
            for t in results:
                t.fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert all(torch.equal(t, v) for t, v in zip(results, want)), i
    torch.cuda.synchronize()


def test_refusals_with_a_plan(plan):
    x, w, out = normal(1, 4, 64), normal(2, 32, 64), torch.empty(4, 32, dtype=BF16, device="cuda")
    bad = [dict(out=torch.empty(4, 40, dtype=BF16, device="cuda")), dict(out=out.half()), dict(x=x.float()), dict(w=w.float()),
           dict(bias=normal(3, 33)), dict(residual=normal(3, 5, 32)), dict(pre=torch.empty(4, 32, device="cuda")),
           dict(x_scale=torch.ones(5, device="cuda")), dict(out=torch.empty(32, 4, dtype=BF16, device="cuda").t()),
           dict(x=x.cpu()), dict(bias=normal(3, 32).cpu()), dict(activation="softmax")]
    for kw in bad:
        args = dict(x=x, w=w, out=out) | kw
        with pytest.raises(ValueError):
            ptg.layer_linear(args.pop("x"), args.pop("w"), args.pop("out"), plan, **args)
    for kw in (dict(x_scale=torch.ones(4, device="cuda")), dict(w_scale=torch.ones(32, device="cuda"))):  # scales of bf16 operands
        with pytest.raises(ptg.PtgError) as e:
            ptg.layer_linear(x, w, out, plan, **kw)
        assert e.value.status == -1
    for shape in ((4, 60), (4, 68)):  # 60: not a multiple of 8 bf16 elements; e4m3 rows need 16
        with pytest.raises(ptg.PtgError) as e:
            ptg.layer_linear(normal(1, *shape), normal(2, 32, shape[1]), out, plan)
        assert e.value.status == -2
    with pytest.raises(ptg.PtgError) as e:
        ptg.layer_linear(normal(1, 4, 72, dtype=E4M3), normal(2, 32, 72, dtype=E4M3), out, plan)
    assert e.value.status == -2
    buf = torch.zeros(4 * 64 + 8, dtype=BF16, device="cuda")
    with pytest.raises(ptg.PtgError) as e:  # misaligned
        ptg.layer_linear(buf[1:257].view(4, 64), w, out, plan)
    assert e.value.status == -1
    with pytest.raises(ptg.PtgError) as e:  # a row stride that breaks the rows' alignment
        ptg.layer_linear(torch.zeros(4, 68, dtype=BF16, device="cuda")[:, :64], w, out, plan)
    assert e.value.status == -2
    with pytest.raises(ptg.PtgError) as e:
        ptg.layer_activation_backward(out, None, out, plan, activation="relu")
    assert e.value.status == -1


def sampled(m, tile, n=24):
    """Rows in every part of the tiles: the first and last, tile borders, and some between."""
    g = torch.Generator().manual_seed(m)
    rows = {0, m - 1, *range(0, m, tile), *range(tile - 1, m, tile)} | set(torch.randint(0, m, (n,), generator=g).tolist())
    return torch.tensor(sorted(r for r in rows if r < m))


# 256 x 256 tiles: whole waves and a split partial one, one partial wave, a long split k; ragged edges and odd k-steps
LARGE = [(4104, 4096, 1032), (1032, 8192, 4096), (520, 8200, 8208), (2049, 4104, 2056)]


@pytest.mark.parametrize("m,n,k", LARGE)
@pytest.mark.parametrize("t", [BF16, E4M3])
def test_linear_large_tiles(plan, m, n, k, t):
    k = k // 16 * 16 if t == E4M3 else k
    say("linear large", m, n, k, t)
    x, w, xs, ws = operands(m, n, k, t)
    b, r = normal(3, n), normal(4, m, n)
    out, z_out = Out(m, n, BF16), Out(m, n, BF16)
    ptg.layer_linear(x, w, out.t, plan, bias=b, activation="silu", residual=r, pre=z_out.t, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    out.check()
    z_out.check()
    assert torch.isfinite(out.t.float()).all()
    rows = sampled(m, 256)
    at = rows.cuda()
    pick = (x.float()[at], w, b, "silu", r[at])
    scales = (None if xs is None else xs[at], ws)
    z, y = ref.linear(pick[0], w, b, "silu", pick[4], *scales)
    bz, by = ref.linear_bounds(pick[0], w, b, "silu", pick[4], BF16, *scales)
    within(out.t[at], y, by, "out")
    within(z_out.t[at], z, bz, "pre")
    again = torch.empty_like(out.t)
    ptg.layer_linear(x, w, again, plan, bias=b, activation="silu", residual=r, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    assert torch.equal(again, out.t), "the same call twice gave different bits"


@pytest.mark.parametrize("m,n,k", LARGE)
def test_linear_backward_large_tiles(plan, m, n, k):
    say("linear backward large", m, n, k)
    dpre, x, w = normal(1, m, n, scale=0.1), normal(2, m, k), normal(3, n, k, scale=k ** -0.5)
    dx, dw = Out(m, k, BF16), Out(n, k, F32)
    ptg.layer_linear_backward(dpre, x, w, plan, dx=dx.t, dw=dw.t)
    torch.cuda.synchronize()
    dx.check()
    dw.check()
    assert torch.isfinite(dx.t.float()).all() and torch.isfinite(dw.t).all()
    at, to = sampled(m, 256).cuda(), sampled(n, 256).cuda()
    within(dx.t[at], *ref.product_bound(dpre[at], w, BF16), "dx")
    within(dw.t[to], *ref.product_bound(dpre.t()[to], x, F32), "dw")


@pytest.mark.parametrize("k", [32, 56, 64, 72, 96, 120, 128, 160, 192, 200, 264, 520])
@pytest.mark.parametrize("m,n", [(130, 264), (300, 520)])
def test_linear_short_and_odd_k(plan, m, n, k):
    """k of one to nine k-steps: pairs of them whole, half empty and cut short, fewer than the ring holds."""
    say("linear short k", m, n, k)
    check_linear(plan, m, n, k)
    check_linear(plan, m, n, (k + 15) // 16 * 16, E4M3, bias=None)
    check_backward(plan, m, k, n)


@pytest.mark.parametrize("m", [1, 17, 130])
def test_linear_strides_that_are_not_looked_at(plan, m):
    """Row strides far past the rows' length, and (one row) any stride at all."""
    x, w = normal(1, m, 136, pad=4096), normal(2, 264, 136, pad=2048)
    if m == 1:
        x = torch.as_strided(x, (1, 136), (3, 1))
    out = Out(m, 264, BF16, pad=512)
    ptg.layer_linear(x, w, out.t, plan)
    torch.cuda.synchronize()
    within(out.t, ref.d(x) @ ref.d(w).t(), ref.linear_bounds(x, w, None, "none", None, BF16)[1], "out")
    out.check()
