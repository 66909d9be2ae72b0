"""The output head's cross entropy and its gradient, which never keep the logits, against the fp64 oracle that does."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests import head_cases
from tests.layer_util import Out, normal, say, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    ptg.layer_sync(p)
    p.destroy()


@pytest.fixture(scope="module")
def streams():
    return torch.cuda.Stream(), torch.cuda.Stream()


def head(m, n, k, pad=0, spread=2.0):
    """x, w and labels: the first and last entries of the vocabulary, entries at the borders of tiles, some not counted."""
    x, w = normal(1, m, k, pad=pad), normal(2, n, k, scale=spread / max(k, 1) ** 0.5, pad=pad)
    g = torch.Generator().manual_seed(m + n)
    label = torch.randint(0, n, (m,), generator=g)
    edges = torch.tensor([0, n - 1, n // 2, min(127, n - 1), min(128, n - 1), min(255, n - 1), min(256, n - 1)])
    label[: len(edges)] = edges[:m]
    if m > 3:
        label[torch.rand(m, generator=g) < 0.2] = -100
        label[3] = -1
    return x, w, label.cuda()


def forward(plan, x, w, label, with_loss=True, **kw):
    m = x.shape[0]
    lse, loss = torch.full((m + 2,), -7.0, device="cuda"), torch.full((m + 2,), -7.0, device="cuda")
    ptg.layer_cross_entropy(x, w, label, lse[1: m + 1], plan, loss=loss[1: m + 1] if with_loss else None, **kw)
    return lse, loss


def check_forward(plan, m, n, k, pad=0, spread=2.0):
    x, w, label = head(m, n, k, pad, spread)
    lse, loss = forward(plan, x, w, label)
    torch.cuda.synchronize()
    assert all(v[0] == -7.0 and v[m + 1] == -7.0 for v in (lse, loss)), "a write outside the output"
    exact, bound = ref.cross_entropy(x, w, label), ref.cross_entropy_bounds(x, w, label)
    within(lse[1: m + 1], exact[0], bound[0], f"lse {m} {n} {k}")
    within(loss[1: m + 1], exact[1], bound[1], f"loss {m} {n} {k}")
    return x, w, label, lse[1: m + 1].clone()


def check_backward(plan, m, n, k, pieces=1, dx_t=BF16, dw_t=BF16, weighted=False, scaled=False, accumulate=False, pad=0, spread=2.0):
    x, w, label, lse = check_forward(plan, m, n, k, pad, spread)
    weight = normal(7, m, dtype=F32) if weighted else None
    dloss = torch.tensor(0.0123, device="cuda") if scaled else None
    old = normal(8, n, k, dtype=dw_t) if accumulate else None
    dx, dw = Out(m, k, dx_t), Out(n, k, dw_t, fill=old)
    size = ptg.layer_cross_entropy_scratch(m, n, k, pieces)
    scratch = torch.full((size + 64,), 96, dtype=torch.uint8, device="cuda")
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch[:size], plan, dx=dx.t, dw=dw.t, weight=weight, dloss=dloss,
                                     accumulate=accumulate)
    torch.cuda.synchronize()
    assert (scratch[size:] == 96).all(), "a write past the scratch"
    dx.check()
    dw.check()
    want = ref.cross_entropy_backward_bounds(x, w, label, lse, dx_t, dw_t, weight, dloss, old)
    within(dx.t, *want[0], f"dx {m} {n} {k}")
    within(dw.t, *want[1], f"dw {m} {n} {k}")
    return dx.t, dw.t


# few rows and tiles; edges inside a tile, a block of columns, a k-step
SHAPES = [(1, 8, 8), (1, 1000, 264), (2, 136, 1032), (5, 5000, 520), (16, 264, 64), (17, 2056, 136), (40, 1032, 264), (64, 520, 2056),
          (65, 8, 8), (66, 136, 40), (100, 264, 520), (128, 1024, 128), (129, 1032, 264), (200, 5000, 72), (257, 520, 264), (300, 2056, 136),
          (600, 3080, 264)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_loss_sizes(plan, m, n, k):
    say("cross entropy", m, n, k)
    check_forward(plan, m, n, k, pad=8)


# vocabularies of any length: ends inside a lane's four columns, its eight, a tile
ODD = [(1, 1, 8), (3, 3, 40), (7, 9, 264), (12, 1001, 136), (24, 16385, 1032), (40, 8197, 2056), (70, 1, 64), (80, 129, 264), (100, 255, 72),
       (150, 511, 520), (300, 257, 136), (260, 1027, 2056), (600, 3086, 264), (1000, 5003, 128)]


@pytest.mark.parametrize("m,n,k", ODD)
def test_any_vocabulary(plan, m, n, k):
    say("any vocabulary", m, n, k)
    check_backward(plan, m, n, k, weighted=True, scaled=True, pad=8)
    if n > 256:
        check_backward(plan, m, n, k, 2, F32, F32, accumulate=True)


# w large enough that few rows' x goes through LDS: one share of k and several, a share that ends inside a segment, a ragged
# last block of w
@pytest.mark.parametrize("m,n,k", [(8, 33032, 1032), (11, 8200, 4104), (16, 2056, 16400), (17, 16392, 1040), (24, 4104, 4112), (32, 2056, 8208),
                                   (33, 8200, 2064), (48, 1032, 32784), (9, 8195, 4104), (30, 2049, 8200), (50, 4102, 4112), (64, 16392, 1296), (63, 4104, 8200)])
def test_loss_of_some_rows_of_a_large_weight(plan, m, n, k):
    say("cross entropy, some rows", m, n, k)
    check_forward(plan, m, n, k, pad=24)
    x, w, label, a = check_forward(plan, m, n, k)
    b = forward(plan, x, w, label)[0][1: m + 1]
    torch.cuda.synchronize()
    assert torch.equal(a, b)


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gradient_sizes(plan, m, n, k):
    say("cross entropy backward", m, n, k)
    check_backward(plan, m, n, k, weighted=True, scaled=True)


@pytest.mark.parametrize("pieces", [1, 2, 3, 100])
@pytest.mark.parametrize("dx_t,dw_t", [(BF16, F32), (F32, BF16)])
def test_gradient_in_pieces(plan, pieces, dx_t, dw_t):
    say("pieces", pieces)
    check_backward(plan, 150, 2056, 264, pieces, dx_t, dw_t, weighted=True, scaled=True, accumulate=True, pad=8)
    check_backward(plan, 70, 1000, 136, pieces, dx_t, dw_t)


def test_gradient_parts(plan):
    m, n, k = 150, 1032, 264
    x, w, label = head(m, n, k)
    lse = forward(plan, x, w, label)[0][1: m + 1]
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k, 2), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    dx2, dw2 = torch.empty_like(dx), torch.empty_like(dw)
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx, dw=dw)
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx2)
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dw=dw2)
    torch.cuda.synchronize()
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    again, only = forward(plan, x, w, label, with_loss=False)
    torch.cuda.synchronize()
    assert torch.equal(again[1: m + 1], lse) and (only == -7.0).all()


@pytest.mark.parametrize("m", [1, 12, 100, 300])
@pytest.mark.parametrize("k", [0, 8])
def test_flat_logits(plan, m, k):
    """Logits that are all alike (k = 0 gives zeros): lse = log n."""
    n = 1032
    x, w = torch.zeros(m, k, dtype=BF16, device="cuda"), torch.ones(n, k, dtype=BF16, device="cuda")
    lse, loss = forward(plan, x, w, torch.arange(m, device="cuda"))
    torch.cuda.synchronize()
    want = torch.log(torch.tensor(float(n), dtype=torch.float64))
    assert (lse[1: m + 1].cpu() - want).abs().max() < 1e-6 and (loss[1: m + 1].cpu() - want).abs().max() < 1e-6


@pytest.mark.parametrize("m", [1, 12, 100, 300])
def test_large_logits(plan, m):
    """Logits of some hundreds, far apart: exponentials vanish or stand alone, and nothing overflows."""
    check_backward(plan, m, 520, 264, spread=200.0)


@pytest.mark.parametrize("m", [4, 40, 100, 300])
def test_labels_not_counted_and_past_the_vocabulary(plan, m):
    n, k = 520, 64
    x, w, _ = head(m, n, k)
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k), dtype=torch.uint8, device="cuda")
    none = torch.full((m,), -100, device="cuda")
    lse, loss = forward(plan, x, w, none)
    dx, dw = torch.full((m, k), 9.0, device="cuda"), torch.full((n, k), 9.0, device="cuda")
    ptg.layer_cross_entropy_backward(x, w, none, lse[1: m + 1], scratch, plan, dx=dx, dw=dw)
    torch.cuda.synchronize()
    assert (loss[1: m + 1] == 0).all() and torch.isfinite(lse).all() and (dx == 0).all() and (dw == 0).all()
    for past in (n, n + 1, 1 << 40):
        label = torch.zeros(m, dtype=torch.int64, device="cuda")
        label[2] = past
        lse, loss = forward(plan, x, w, label)
        ptg.layer_cross_entropy_backward(x, w, label, lse[1: m + 1], scratch, plan, dx=dx)
        torch.cuda.synchronize()
        bad = torch.arange(m, device="cuda") == 2
        assert torch.equal(torch.isnan(loss[1: m + 1]), bad) and torch.isfinite(lse).all(), past
        assert torch.equal(torch.isnan(dx).all(dim=1), bad) and torch.equal(torch.isnan(dx).any(dim=1), bad), past


@pytest.mark.parametrize("m", [4, 40, 100, 300])
def test_non_finite_logits(plan, m):
    """NaN in a row of x stays in that row, and a row that is not counted, or weighs nothing, gives dz = 0 with it; entries
    of the vocabulary that are masked by -infinity have no part; an infinite logit takes all."""
    n, k = 520, 64
    x, w, label = head(m, n, k)
    x[:, 0], w[:, 0] = 1.0, 0.0
    w[5], w[200: 400] = 0.0, 0.0
    w[5, 0], w[200: 400, 0] = -float("inf"), -float("inf")  # a whole block of columns among them
    label[:] = 0
    label[1] = -100
    lse, loss = forward(plan, x, w, label)
    torch.cuda.synchronize()
    z = x.double().cpu() @ torch.where(torch.isinf(w), torch.zeros_like(w), w).double().cpu().t()
    z[:, 5], z[:, 200: 400] = -float("inf"), -float("inf")
    want = torch.logsumexp(z, dim=1)
    assert (lse[1: m + 1].cpu() - want).abs().max() < 1e-4
    y, v, _ = head(m, n, k)
    lse = forward(plan, y, v, label)[0][1: m + 1]
    y[1, 3], y[2, 3] = float("nan"), float("nan")
    bad_lse, bad_loss = forward(plan, y, v, label)
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k), dtype=torch.uint8, device="cuda")
    weight = torch.ones(m, device="cuda")
    weight[2] = 0.0
    dx, dx_all = torch.empty(m, k, device="cuda"), torch.empty(m, k, device="cuda")
    ptg.layer_cross_entropy_backward(y, v, label, lse, scratch, plan, dx=dx, weight=weight)
    ptg.layer_cross_entropy_backward(y, v, label, lse, scratch, plan, dx=dx_all)
    torch.cuda.synchronize()
    nan = torch.isnan(bad_lse[1: m + 1])
    assert nan[1] and nan[2] and int(nan.sum()) == 2
    assert bad_loss[2] == 0 and torch.isnan(bad_loss[3]) and torch.isfinite(bad_loss[1]) and torch.isfinite(bad_loss[4: m + 1]).all()
    assert (dx[1] == 0).all() and (dx[2] == 0).all() and torch.isfinite(dx).all()
    assert (dx_all[1] == 0).all() and torch.isnan(dx_all[2]).all() and torch.isfinite(dx_all[3:]).all() and torch.isfinite(dx_all[0]).all()


def test_rows_in_several_runs(plan):
    """So large a vocabulary that the workspace holds the blocks' sums of a part of the rows only."""
    m, n, k = 1300, 1 << 20, 8
    x, w, label = head(m, n, k)
    lse, loss = forward(plan, x, w, label)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 255, 256, 511, 512, 767, 768, 1023, 1024, 1279, 1280, 1299]).cuda()
    exact, bound = ref.cross_entropy(x[at], w, label[at]), ref.cross_entropy_bounds(x[at], w, label[at])
    within(lse[1:-1][at], exact[0], bound[0], "lse")
    within(loss[1:-1][at], exact[1], bound[1], "loss")
    assert torch.isfinite(lse).all() and torch.isfinite(loss).all()


def test_empty_batches(plan):
    x, w = torch.empty(0, 64, dtype=BF16, device="cuda"), normal(1, 264, 64)
    label, v, s = torch.empty(0, dtype=torch.int64, device="cuda"), torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda")
    dw = torch.full((264, 64), 9.0, device="cuda")
    ptg.layer_cross_entropy(x, w, label, v, plan, loss=torch.empty(0, device="cuda"))
    ptg.layer_cross_entropy_backward(x, w, label, v, s, plan, dw=dw, accumulate=True)
    torch.cuda.synchronize()
    assert (dw == 9.0).all()
    ptg.layer_cross_entropy_backward(x, w, label, v, s, plan, dx=torch.empty_like(x), dw=dw, dloss=torch.tensor(float("inf"), device="cuda"))
    torch.cuda.synchronize()
    assert (dw == 0).all()


def test_gradient_against_differences(plan):
    """Along random directions, the gradient against central differences of the loss in 64 bits, off by the roundings of dz
    (2^-8 of each) and of lse (some 2^-20)."""
    m, n, k = 40, 264, 136
    x, w, label = head(m, n, k)
    weight, dloss = normal(7, m, dtype=F32), torch.tensor(0.3, device="cuda")
    lse = forward(plan, x, w, label)[0][1: m + 1]
    dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k), dtype=torch.uint8, device="cuda")
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx, dw=dw, weight=weight, dloss=dloss)
    torch.cuda.synchronize()
    for seed in range(4):
        u, v = ref.d(normal(20 + seed, m, k, dtype=F32)), ref.d(normal(30 + seed, n, k, dtype=F32))
        h = 1e-5
        loss = lambda t: 0.3 * (ref.d(weight) * ref.cross_entropy(ref.d(x) + t * u, ref.d(w) + t * v, label)[1]).sum()  # noqa: E731
        diff = (loss(h) - loss(-h)) / (2 * h)
        got = (ref.d(dx) * u).sum() + (ref.d(dw) * v).sum()
        dz = ref.logit_grad(x, w, label, lse, weight).abs()
        along = u.abs() @ ref.d(w).abs().t() + ref.d(x).abs() @ v.abs().t()
        size = 0.3 * (dz * along).sum() * (2.0 ** -8 + 2.0 ** -12)
        assert abs(diff - got) <= size, (float(diff), float(got), float(size))


def test_calls_on_two_streams_are_ordered(plan, streams):
    m, n, k = 200, 1032, 264
    x, w, label = head(m, n, k)
    scratch = [torch.empty(ptg.layer_cross_entropy_scratch(m, n, k, 2), dtype=torch.uint8, device="cuda") for _ in range(2)]

    def step(stream, scratch):
        lse, loss = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
        dx, dw = torch.empty(m, k, device="cuda"), torch.empty(n, k, device="cuda")
        few, few_loss = torch.empty(12, device="cuda"), torch.empty(12, device="cuda")
        torch.cuda.synchronize()
        ptg.layer_cross_entropy(x, w, label, lse, plan, loss=loss, stream=stream)
        ptg.layer_cross_entropy(x[:12], w, label[:12], few, plan, loss=few_loss, stream=stream)
        ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx, dw=dw, stream=stream)
        return lse, loss, few, few_loss, dx, dw

    want = step(None, scratch[0])
    torch.cuda.synchronize()
    outs = [step(streams[i % 2], scratch[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    ptg.layer_sync(plan)


@pytest.mark.parametrize("m", [12, 100, 300])
def test_a_step_replays_from_a_graph(plan, streams, m):
    """Loss and gradient captured once and replayed over changing inputs, with the plan's own uncaptured calls between."""
    n, k = 1032, 264
    x, w, label = head(m, n, k)
    lse, loss = torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    dx, dw = torch.empty(m, k, dtype=BF16, device="cuda"), torch.zeros(n, k, device="cuda")
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k, 2), dtype=torch.uint8, device="cuda")
    dloss = torch.tensor(0.01, device="cuda")

    def step():
        ptg.layer_cross_entropy(x, w, label, lse, plan, loss=loss)
        ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx, dw=dw, dloss=dloss)

    results = (lse, loss, dx, dw)
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
            dloss.fill_(0.01 * (i + 1))
            step()
            s.synchronize()
            want = [t.clone() for t in results]
            for t in results:
                t.fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert all(torch.equal(t, v) for t, v in zip(results, want)), i
    torch.cuda.synchronize()


def check_sampled(plan, m, n, k, pieces=1, backward=True):
    """Some rows of every output against the oracle, the whole of it finite and the same bits twice."""
    x, w, label = head(m, n, k)
    lse, loss = forward(plan, x, w, label)
    at = torch.randperm(m, generator=torch.Generator().manual_seed(m))[:40]
    at = torch.cat([at, torch.tensor([0, 255, 256, m - 1]).clamp(max=m - 1)]).cuda()
    torch.cuda.synchronize()
    exact, bound = ref.cross_entropy(x[at], w, label[at]), ref.cross_entropy_bounds(x[at], w, label[at])
    within(lse[1:-1][at], exact[0], bound[0], f"lse {m} {n} {k}")
    within(loss[1:-1][at], exact[1], bound[1], f"loss {m} {n} {k}")
    again = forward(plan, x, w, label)
    torch.cuda.synchronize()
    assert torch.equal(again[0], lse) and torch.equal(again[1], loss) and torch.isfinite(lse).all() and torch.isfinite(loss).all()
    if not backward:
        return
    dx, dw = Out(m, k, BF16), Out(n, k, F32)
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, k, pieces), dtype=torch.uint8, device="cuda")
    ptg.layer_cross_entropy_backward(x, w, label, lse[1: m + 1], scratch, plan, dx=dx.t, dw=dw.t)
    torch.cuda.synchronize()
    dx.check()
    dw.check()
    (want, off), _ = ref.cross_entropy_backward_bounds(x[at], w, label[at], lse[1:-1][at], BF16, F32)
    within(dx.t[at], want, off, f"dx {m} {n} {k}")
    # dw's rows: dz's columns of some of the vocabulary's entries
    to = torch.randperm(n, generator=torch.Generator().manual_seed(n))[:40]
    to = torch.cat([to, torch.tensor([0, 255, 256, n - 1]).clamp(max=n - 1)]).cuda()
    z, v = ref.d(x) @ ref.d(w[to]).t(), ref.d(lse[1:-1])[:, None]
    dz = torch.exp(z - v) - (label.cpu()[:, None] == to.cpu()[None, :]).double()
    dz[label.cpu() < 0] = 0.0
    t = ref._logits_error(x, w[to]) + 3 * ref.U32 * (z.abs() + v.abs())
    err = torch.exp(z - v) * (torch.expm1(t) + 4 * ref.U32) + 2 * ref.U32
    err = err + 2.0 ** -8 * (dz.abs() + err) + 2.0 ** -126
    exact_dw = dz.t() @ ref.d(x)
    off = ref.rounded(exact_dw, F32, err.t() @ ref.d(x).abs() + (dz.abs().t() @ ref.d(x).abs()) * (m + 64) * ref.U32)
    within(dw.t[to], exact_dw, off, f"dw {m} {n} {k}")
    dx2, dw2 = torch.empty_like(dx.t), torch.empty_like(dw.t)
    ptg.layer_cross_entropy_backward(x, w, label, lse[1: m + 1], scratch, plan, dx=dx2, dw=dw2)
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx.t) and torch.equal(dw2, dw.t) and torch.isfinite(dx2).all() and torch.isfinite(dw2).all()


# whole waves of 256 x 256 tiles and a split partial one; ragged edges; long k; several pieces
LARGE = [(1000, 8200, 2056, 1), (520, 33032, 1032, 3), (2049, 4104, 520, 1), (260, 16392, 4104, 2)]


@pytest.mark.parametrize("m,n,k,pieces", LARGE)
def test_large(plan, m, n, k, pieces):
    say("cross entropy large", m, n, k)
    check_sampled(plan, m, n, k, pieces)


@pytest.mark.parametrize("what,kind,m,n,k", [c for c in head_cases.CASES if c[1] != "i8"])
def test_every_kernel(plan, what, kind, m, n, k):
    say(what, kind, m, n, k)
    check_sampled(plan, m, n, k, backward=kind != "loss")


def test_refusals(plan):
    x, w, label = head(8, 64, 32)
    lse, s = torch.empty(8, device="cuda"), torch.empty(4096, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    good = dict(x=x, w=w, label=label, lse=lse)
    for kw in (dict(x=x.float()), dict(w=w.float()), dict(w=normal(2, 64, 40)), dict(label=label.int()), dict(label=label[:7]),
               dict(label=label.cpu()), dict(lse=lse[:7]), dict(lse=lse.double()), dict(x=x.t()), dict(label=torch.zeros(16, dtype=torch.int64, device="cuda")[::2])):
        a = good | kw
        with pytest.raises(ValueError):
            ptg.layer_cross_entropy(a["x"], a["w"], a["label"], a["lse"], plan)
        with pytest.raises(ValueError):
            ptg.layer_cross_entropy_backward(a["x"], a["w"], a["label"], a["lse"], s, plan, dx=dx)
    for kw in (dict(dx=dx[:7]), dict(dw=dx), dict(dx=dx, weight=lse[:7]), dict(dx=dx, dloss=lse), dict(dx=dx, dloss=lse[0].double()), dict()):
        with pytest.raises(ValueError):
            ptg.layer_cross_entropy_backward(x, w, label, lse, s, plan, **kw)
    for scratch in (s[:512], s[8: 2048]):  # too small, misaligned
        with pytest.raises(ptg.PtgError):
            ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx)
    with pytest.raises(ValueError):
        ptg.layer_cross_entropy_backward(x, w, label, lse, s.cpu(), plan, dx=dx)
    with pytest.raises(ptg.PtgError):
        ptg.layer_cross_entropy(x, w, label, lse, plan, loss=lse)
