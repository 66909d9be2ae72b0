"""Relative accuracy of the activations and their gradients, the far tails included, against 64 bits.

The argument z reaches the activation exactly: x is zero and z is the fp32 bias, the output fp32. The gradient comes out
in fp32 as dbias of one row.

Bounds, in units u = 2^-24 (the instructions' results are off by one unit in the last place, 2 u): an exponential 4 u (its
instruction and two roundings), a reciprocal 2 u, every other operation u. silu: 1 + e, its reciprocal and the last product,
4 u after the exponential's 4. gelu: the two polynomials of positive terms at most 9 and 11 u, reciprocal, three products,
the fit's 0.1 u: 30 u with the exponential, and the last product. tanh-gelu: its logistic's argument t = 2 c z (1 + a z^2)
takes five roundings and its product with log2 e one and a quarter, which the exponential turns into 6.25 |t| u of the result. Below 2^-126, the smallest normal number,
results may become zero: one argument's worth of that is allowed.
"""

import math

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import say, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


@pytest.fixture(scope="module")
def plan():
    p = ptg.layer_create()
    yield p
    p.destroy()


def arguments():
    """Tails as far as the results are normal numbers, the region around zero, and tiny arguments."""
    z = torch.cat([torch.linspace(-13.0, 9.0, 20001), torch.linspace(-87.0, 20.0, 10001), torch.logspace(-12, 0, 1499),
                   -torch.logspace(-12, 0, 1499)]).to(F32)
    return torch.cat([z, torch.zeros(-len(z) % 8)])


def gelu_cdf(z):
    return torch.special.erfc(-z / math.sqrt(2)) / 2


def tanh_argument(z):
    return 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)


def exact(z, act):
    if act == "gelu":
        return z * gelu_cdf(z)
    return z / (1 + torch.exp(-(tanh_argument(z) if act == "gelu_tanh" else z)))


def units(z, act):
    if act == "gelu":
        return torch.full_like(z, 31.0)
    return 9.0 + (6.25 * tanh_argument(z).abs() if act == "gelu_tanh" else 0 * z)


@pytest.mark.parametrize("m,k", [(1, 64), (1, 0), (300, 64), (130, 8192)])  # few rows, no sum at all, whole tiles, split ones
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_keep_their_relative_accuracy(plan, m, k, act):
    say("activation accuracy", m, k, act)
    bias = arguments().cuda()
    n = len(bias)
    if k == 8192:
        bias, n = bias[::32].contiguous()[: len(bias) // 256 * 8], len(bias) // 256 * 8
    out = torch.empty(m, n, device="cuda")
    ptg.layer_linear(torch.zeros(m, k, dtype=BF16, device="cuda"), torch.zeros(n, k, dtype=BF16, device="cuda"), out, plan, bias=bias,
                     activation=act)
    torch.cuda.synchronize()
    z = ref.d(bias)
    y = exact(z, act)
    bound = y.abs() * units(z, act) * U + 2.0 ** -126 * z.abs().clamp(min=1)
    within(out[0], y, bound, act)
    assert all(torch.equal(out[0], out[i]) for i in range(1, m, 37))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activation_gradients_keep_their_accuracy(plan, act):
    """Each term of f'(z) = p + z p' to its own accuracy: 31 u and the formulas' further roundings (three products of the
    second term, for gelu_tanh 6.25 |t| u in p and twice that in p (1 - p), whose 1 - p is off by a rounding of p, and the last sum)."""
    z = arguments().to(BF16).cuda()
    db = torch.empty(len(z), device="cuda")
    ptg.layer_activation_backward(torch.ones(1, len(z), dtype=BF16, device="cuda"), z[None], None, plan, activation=act, dbias=db)
    torch.cuda.synchronize()
    v = ref.d(z)
    want = ref.act_grad(v, act)
    if act == "gelu":
        p, q, slack = gelu_cdf(v), torch.exp(-v * v / 2) / math.sqrt(2 * math.pi), 36.0
        loss = 0 * v
    else:
        t = tanh_argument(v) if act == "gelu_tanh" else v
        p = 1 / (1 + torch.exp(-t))
        slope = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * v * v) if act == "gelu_tanh" else torch.ones_like(v)
        want = p + v * slope * p / (1 + torch.exp(t))
        q, slack = slope * p / (1 + torch.exp(t)), 16.0 + (18.75 * t.abs() if act == "gelu_tanh" else 0 * t)
        loss = (v * slope * p).abs() * 9 * U  # 1 - p, from a p that is off by 9 u and rounded
    bound = (p + (v * q).abs()) * slack * U + loss + 2.0 ** -126 * v.abs().clamp(min=1) ** 3
    within(db, want, bound, act)
