"""Every kernel of the products, split and way of running them against the oracle: the cases of layer_cases.py, of which
test_layer_dispatch.py asserts what they run.

Sampled rows and columns (every tile's edges among them) are compared with 64 bits; the whole output with the same formula
in fp32 by torch, whose sums may be off by as much again as the kernel's."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests import layer_cases
from tests.layer_util import Out, say, within

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    ptg.layer_sync(p)
    p.destroy()


def normal(seed, *shape, scale=1.0, dtype=BF16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def sampled(n, most=160):
    """The first and last indexes, those at every 128-wide border (or an even choice of them), and some between."""
    borders = [i for b in range(0, n, 128) for i in (b - 1, b) if 0 <= i < n]
    if len(borders) > most:
        borders = borders[:: len(borders) // most + 1]
    some = torch.randint(0, n, (24,), generator=torch.Generator().manual_seed(n)).tolist()
    return torch.tensor(sorted({0, n - 1, *borders, *some}), device="cuda")


def whole(got, want, size, k, dtype, slope=1.0, extra=0.0):
    """got against fp32 values: both sums may be off by (k + 8) u of the sum of magnitudes."""
    bound = 2 * slope * size * (k + 8) * ref.U32 + extra + ref.HALF_STEP[dtype] * want.abs() * 1.01 + ref.TINY[dtype]
    bad = ~((got.float() - want).abs() <= bound)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} values off, first at {bad.nonzero()[0].tolist()}"


@pytest.mark.parametrize("runs,t,m,n,k", layer_cases.LINEAR, ids=[c[0] + " " + c[1] for c in layer_cases.LINEAR])
def test_linear(plan, runs, t, m, n, k):
    say("linear", runs, m, n, k)
    t = {"bf16": BF16, "e4m3": E4M3}[t]
    xs = ws = None
    if t == E4M3:
        x, w = normal(1, m, k, scale=60.0, dtype=E4M3), normal(2, n, k, scale=60.0, dtype=E4M3)
        xs, ws = 0.001 + 0.02 * normal(5, m, dtype=F32).abs(), (0.001 + 0.02 * normal(6, n, dtype=F32).abs()) / k ** 0.5
    else:
        x, w = normal(1, m, k), normal(2, n, k, scale=k ** -0.5)
    b, r = normal(3, n), normal(4, m, n)
    out, pre = Out(m, n, F32), Out(m, n, BF16)
    ptg.layer_linear(x, w, out.t, plan, bias=b, activation="silu", residual=r, pre=pre.t, x_scale=xs, w_scale=ws)
    again = torch.empty(m, n, device="cuda")
    ptg.layer_linear(x, w, again, plan, bias=b, activation="silu", residual=r, x_scale=xs, w_scale=ws)
    torch.cuda.synchronize()
    out.check()
    pre.check()
    assert torch.equal(again, out.t), "the same call twice gave different bits"
    at, to = sampled(m), sampled(n)

    def pick(v, i):
        return None if v is None else v[i]

    def rows(v, i):  # (indexing is not there for e4m3)
        return v.float()[i]

    part = (rows(x, at), rows(w, to), b[to], "silu", r[at][:, to], pick(xs, at), pick(ws, to))
    z, y = ref.linear(*part)
    bz, by = ref.linear_bounds(*part[:5], F32, *part[5:])
    within(out.t[at][:, to], y, by, "out")
    within(pre.t[at][:, to], z, bz, "pre")
    scale = 1.0 if xs is None else xs[:, None] * ws
    z, size = torch.matmul(x.float(), w.float().t()) * scale + b.float(), torch.matmul(x.float().abs(), w.float().abs().t()) * scale + b.float().abs()
    whole(pre.t, z, size, k, BF16)
    whole(out.t, torch.nn.functional.silu(z) + r.float(), size, k, F32, 1.2, 2.0 ** -20 * (z.abs() + r.float().abs()))


@pytest.mark.parametrize("runs,kind,m,n,k", layer_cases.BACKWARD, ids=[c[0] for c in layer_cases.BACKWARD])
def test_linear_backward(plan, runs, kind, m, n, k):
    say("linear backward", runs, m, n, k)
    dpre = normal(1, m, n, scale=0.1)
    if kind == "dx":
        b, shape, dtype, sums = normal(3, n, k, scale=k ** -0.5), (m, k), BF16, n
        a = dpre
        call = lambda o: ptg.layer_linear_backward(dpre, None, b, plan, dx=o)  # noqa: E731
    else:
        b, shape, dtype, sums = normal(2, m, k), (n, k), F32, m
        a = dpre.t()
        call = lambda o: ptg.layer_linear_backward(dpre, b, None, plan, dw=o)  # noqa: E731
    out, again = Out(*shape, dtype), torch.empty(*shape, dtype=dtype, device="cuda")
    call(out.t)
    call(again)
    torch.cuda.synchronize()
    out.check()
    assert torch.equal(again, out.t), "the same call twice gave different bits"
    at, to = sampled(shape[0]), sampled(shape[1])
    within(out.t[at][:, to], *ref.product_bound(a[at], b[:, to], dtype), kind)
    af = a.float().contiguous()
    whole(out.t, torch.matmul(af, b.float()), torch.matmul(af.abs(), b.float().abs()), sums, dtype)
