"""8-bit rows, their product and the output head's cross entropy without a GPU: the oracle against differences and closed
forms, and every refusal that needs no device."""

import ctypes

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from persistent_tiled_gemm_amd import layer
from tests import hip_stand_in

INVALID, SHAPE = -1, -2
P = 0x100000


def rand(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


def test_oracle_cross_entropy_is_torchs():
    x, w, label = rand(9, 24, seed=1), rand(40, 24, seed=2), torch.tensor([0, 39, -100, 7, 7, 1, -1, 3, 20])
    lse, loss = ref.cross_entropy(x, w, label)
    want = torch.nn.functional.cross_entropy(x @ w.t(), torch.where(label < 0, torch.full_like(label, -100), label), reduction="none")
    assert (loss - want).abs().max() < 1e-12 and (lse - torch.logsumexp(x @ w.t(), dim=1)).abs().max() < 1e-12
    assert torch.isnan(ref.cross_entropy(x, w, torch.full((9,), 40))[1]).all()


def test_oracle_cross_entropy_gradient_is_its_difference():
    m, n, k = 7, 24, 16
    x, w, label, weight = rand(m, k, seed=1), rand(n, k, seed=2), torch.tensor([0, 23, -100, 5, 5, -1, 11]), rand(m, seed=3)
    dloss = torch.tensor(0.37, dtype=torch.float64)
    dx, dw = ref.cross_entropy_backward(x, w, label, ref.cross_entropy(x, w, label)[0], weight, dloss)
    h = 1e-6
    for seed in range(4):
        u, v = rand(m, k, seed=10 + seed), rand(n, k, seed=20 + seed)
        loss = lambda t: dloss * (weight * ref.cross_entropy(x + t * u, w + t * v, label)[1]).sum()  # noqa: E731
        assert abs((loss(h) - loss(-h)) / (2 * h) - ((dx * u).sum() + (dw * v).sum())) < 1e-7


def test_oracle_quantise_rows():
    x = torch.tensor([[0.0, -0.0], [127.0, -63.5], [2.0, 1.0], [float("inf"), 1.0], [1.0, float("nan")]])
    scale, codes = ref.quantise_rows(x, torch.int8)
    assert scale[:2].tolist() == [1.0, 1.0] and codes[:2].tolist() == [[0, 0], [127, -64]]
    assert codes[2].tolist() == [127, 64] and torch.isnan(scale[3:]).all() and (codes[3:] == 0).all()
    scale, codes = ref.quantise_rows(x, torch.float8_e4m3fn)
    assert codes[1].float().tolist() == [448.0, -224.0] and torch.isnan(codes[3:].float()).all()


def call_quantize(**kw):
    a = layer.QuantizeArgs(x=P, out=P, scale=P, m=4, n=64, ldx=64, ldo=64, type=1, out_type=3)
    for k, v in kw.items():
        setattr(a, k, v)
    return layer._library().layer_quantize(ctypes.byref(a), None)


@pytest.mark.parametrize("kw,status", [
    (dict(type=2), INVALID), (dict(type=3), INVALID), (dict(out_type=0), INVALID), (dict(out_type=1), INVALID), (dict(out_type=4), INVALID),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(scale=None), INVALID), (dict(x=P + 8), INVALID), (dict(out=P + 8), INVALID),
    (dict(scale=P + 2), INVALID), (dict(n=60), SHAPE), (dict(n=-8), SHAPE), (dict(m=-1), SHAPE), (dict(m=(1 << 30) + 1), SHAPE),
    (dict(n=(1 << 20) + 8, ldx=1 << 21, ldo=1 << 21), SHAPE), (dict(ldx=56), SHAPE), (dict(ldo=68), SHAPE), (dict(ldx=(1 << 20) + 8), SHAPE)])
def test_quantize_refuses(kw, status):
    assert call_quantize(**kw) == status


def test_empty_quantize_is_accepted_without_a_device():
    assert call_quantize(m=0, x=None, out=None, scale=None) == 0
    assert call_quantize(n=0, x=None, out=None, scale=None) == 0


def test_null_structs_and_plans_are_refused():
    lib = layer._library()
    assert lib.layer_quantize(None, None) == INVALID
    for f, cls in ((lib.layer_cross_entropy, layer.CrossEntropyArgs), (lib.layer_cross_entropy_backward, layer.CrossEntropyGradArgs)):
        assert f(None, None, None) == INVALID
        assert f(ctypes.byref(cls()), None, None) == INVALID


@pytest.fixture(scope="module")
def stand_in(tmp_path_factory):
    return hip_stand_in.built(tmp_path_factory.mktemp("stand_in"))


LOSS = "layer.CrossEntropyArgs(**(dict(x=P, w=P, label=P, lse=P, loss=2 * P, m=4, n=64, k=32, ldx=32, ldw=32) | kw))"
GRAD = ("layer.CrossEntropyGradArgs(**(dict(x=P, w=P, label=P, lse=P, weight=P, dloss=P, dx=P, dw=P, scratch=P, scratch_bytes=512, m=4, "
        "n=64, k=32, ldx=32, ldw=32, lddx=32, lddw=32, dx_type=1, dw_type=1) | kw))")
BOTH = [(dict(x=None), INVALID), (dict(w=None), INVALID), (dict(label=None), INVALID), (dict(lse=None), INVALID), (dict(x=P + 8), INVALID),
        (dict(w=P + 2), INVALID), (dict(label=P + 4), INVALID), (dict(lse=P + 2), INVALID), (dict(m=-1), SHAPE), (dict(n=0), SHAPE),
        (dict(n=-1), SHAPE), (dict(k=28), SHAPE), (dict(n=(1 << 20) + 1), SHAPE), (dict(k=(1 << 20) + 8), SHAPE), (dict(ldx=24), SHAPE),
        (dict(ldw=36), SHAPE), (dict(m=(1 << 30) + 1), SHAPE)]


def statuses(stand_in, function, args, cases):
    return hip_stand_in.run(stand_in, f"""
assert lib.layer_create(ctypes.byref(plan), 0) == 0
hip.stand_in_launches()
result = [[call(lib.{function}, {args}), len(hip.stand_in_launches())] for kw in {cases!r}]
""")


def test_cross_entropy_refuses(stand_in):
    cases = BOTH + [(dict(loss=2 * P + 2), INVALID), (dict(loss=P), INVALID)]
    got = statuses(stand_in, "layer_cross_entropy", LOSS, [c[0] for c in cases])
    assert got == [[s, 0] for _, s in cases]  # refused, and nothing launched
    ok = [dict(m=0, x=None, w=None, label=None, lse=None), dict(m=0, n=0)]
    assert statuses(stand_in, "layer_cross_entropy", LOSS, ok) == [[0, 0]] * 2
    got = statuses(stand_in, "layer_cross_entropy", LOSS, [dict(), dict(loss=None), dict(k=0, x=None, w=None), dict(m=1, ldx=3), dict(n=1), dict(n=61)])
    assert all(s == 0 and n > 0 for s, n in got)


def test_cross_entropy_backward_refuses(stand_in):
    cases = BOTH + [(dict(weight=P + 2), INVALID), (dict(dloss=P + 2), INVALID), (dict(dx=P + 8), INVALID), (dict(dw=P + 8), INVALID),
                    (dict(scratch=P + 8), INVALID), (dict(scratch=None), INVALID), (dict(dx_type=2), INVALID), (dict(dw_type=3), INVALID),
                    (dict(accumulate=2), INVALID), (dict(accumulate=-1), INVALID), (dict(lddx=24), SHAPE), (dict(lddw=28), SHAPE),
                    (dict(scratch_bytes=-1), SHAPE), (dict(scratch_bytes=511), SHAPE), (dict(scratch_bytes=0), SHAPE),
                    # a piece of 256, but no room for dx's sum; the sum, but no piece
                    (dict(n=1024, scratch_bytes=2048), SHAPE), (dict(n=1024, scratch_bytes=2048 + 511), SHAPE),
                    # dz's rows are of whole 8s
                    (dict(n=61, scratch_bytes=2 * 4 * 61), SHAPE), (dict(n=61, scratch_bytes=511), SHAPE)]
    got = statuses(stand_in, "layer_cross_entropy_backward", GRAD, [c[0] for c in cases])
    assert got == [[s, 0] for _, s in cases]
    ok = [dict(m=0, x=None, w=None, label=None, lse=None, dw=None, scratch=None, scratch_bytes=0), dict(m=0, accumulate=1, scratch=None),
          dict(dx=None, dw=None), dict(k=0)]
    assert statuses(stand_in, "layer_cross_entropy_backward", GRAD, ok) == [[0, 0]] * 4
    runs = [dict(), dict(weight=None, dloss=None), dict(n=1024, scratch_bytes=2048 + 512), dict(n=1024, dx_type=0, scratch_bytes=2048),
            dict(n=1024, dx=None, scratch_bytes=2048), dict(m=0, scratch=None, scratch_bytes=0, dx=None), dict(n=61), dict(n=1), dict(n=1021, scratch_bytes=2048 + 512)]
    got = statuses(stand_in, "layer_cross_entropy_backward", GRAD, runs)
    assert all(s == 0 and n > 0 for s, n in got)


def test_int8_product_refuses_what_its_sums_do_not_hold(stand_in):
    line = "layer.LinearArgs(**(dict(x=P, w=P, out=P, m=4, n=64, k=64, ldx=1 << 20, ldw=1 << 20, ldo=64, in_type=3, out_type=1) | kw))"
    cases = [(dict(k=131056), 0), (dict(k=131072), SHAPE), (dict(k=72), SHAPE), (dict(in_type=4), INVALID), (dict(x_scale=P + 8), INVALID)]
    assert [s for s, _ in statuses(stand_in, "layer_linear", line, [c[0] for c in cases])] == [s for _, s in cases]


@pytest.mark.parametrize("m,n,k", [(1, 8, 8), (1000, 50264, 2056), (4096, 131072, 4096), (7, 1 << 20, 64), (0, 64, 64), (3, 1, 8), (300, 50257, 768), (5, 1021, 64)])
def test_scratch_sizes(m, n, k):
    whole = -(-n // 8) * 8
    for pieces in (1, 2, 3, 7, 64, 100000):
        size = ptg.layer_cross_entropy_scratch(m, n, k, pieces)
        sums = 0 if size == 2 * m * whole else 4 * m * k
        piece = whole if m == 0 else (size - sums) // (2 * m)
        assert -(-n // piece) <= pieces or piece == 256 or pieces > n // 256
        assert piece == whole or piece % 256 == 0
    for bad in ((-1, 64, 64, 1), (4, -1, 64, 1), (4, (1 << 20) + 1, 64, 1), (4, 64, 60, 1), (4, 64, 64, 0)):
        with pytest.raises(ValueError):
            ptg.layer_cross_entropy_scratch(*bad)


def test_binding_refuses_host_tensors():
    x, w, v, i = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16), torch.zeros(2), torch.zeros(2, dtype=torch.int64)

    class Plan:
        handle, device = None, 0
    with pytest.raises(ValueError):
        ptg.layer_quantize(x, x.to(torch.int8), v)
    with pytest.raises(ValueError):
        ptg.layer_cross_entropy(x, w, i, v, Plan())
    with pytest.raises(ValueError):
        ptg.layer_cross_entropy_backward(x, w, i, v, v, Plan(), dx=x)
    with pytest.raises(ValueError):
        ptg.layer_cross_entropy_backward(x, w, i, v, v, Plan())
