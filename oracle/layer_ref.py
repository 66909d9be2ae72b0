"""fp64 definitions of the layer operators and the error bounds their kernels are held to.

Inputs are torch tensors of any float type (on the CPU); everything is computed in float64. The bounds count what
the operators' contract allows: fp32 arithmetic (each operation off by at most 2^-24 relative, an fp32 sum of n
terms by at most n 2^-24 of the sum of their magnitudes) and one rounding to the output's type (half a step).
"""

from __future__ import annotations

import math

import torch

U32 = 2.0 ** -24  # half a step of fp32
E4M3_MAX = 448.0
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
# half the smallest subnormal step: what is lost near zero
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float8_e4m3fn: 2.0 ** -10}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def d(t):
    return None if t is None else t.detach().to("cpu").to(torch.float64)


def act(z, name):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2)) / 2
    if name == "gelu_tanh":
        return z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))) / 2
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z.clone()


def act_grad(z, name):
    if name == "relu":
        return torch.where(z > 0, 1.0, 0.0).to(torch.float64)
    if name == "gelu":
        return torch.special.erfc(-z / math.sqrt(2)) / 2 + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return (1 + t) / 2 + z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z) / 2
    if name == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def rmsnorm(x, weight, residual=None, eps=1e-6):
    """(s, y) of the norm."""
    s = d(x) if residual is None else d(x) + d(residual)
    y = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    return s, y if weight is None else y * d(weight)


def quantise(y):
    """(scale, y / scale) of e4m3 rows, before the codes' rounding."""
    top = y.abs().amax(dim=1)
    scale = torch.where(top == 0, torch.ones_like(top), (top / E4M3_MAX).clamp(min=2.0 ** -126))
    return scale, y / scale[:, None]


def rmsnorm_backward(dy, s, weight, dsum=None, eps=1e-6):
    """(dx, dweight)."""
    dy, s = d(dy), d(s)
    r = 1 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    h = s * r
    g = dy if weight is None else dy * d(weight)
    dx = r * (g - h * (g * h).mean(dim=1, keepdim=True))
    return dx if dsum is None else dx + d(dsum), (dy * h).sum(dim=0)


def linear(x, w, bias=None, activation="none", residual=None, x_scale=None, w_scale=None):
    """(z, out)."""
    z = d(x) @ d(w).t()
    if x_scale is not None:
        z = z * d(x_scale)[:, None]
    if w_scale is not None:
        z = z * d(w_scale)[None, :]
    if bias is not None:
        z = z + d(bias)
    y = act(z, activation)
    return z, y if residual is None else y + d(residual)


# ---- bounds: |got - exact| <= bound, element by element

def rounded(exact, dtype, err):
    """A value within `err` of exact, rounded once to dtype."""
    return err + HALF_STEP[dtype] * (exact.abs() + err) + TINY[dtype]


def rmsnorm_bound(y, dtype, n):
    # the sum of squares: terms and a chain of at most 64 additions a thread, then the tree; its root halves
    # that; then a handful of products
    return rounded(y, dtype, y.abs() * (64 + 16) * U32)


def rmsnorm_backward_bounds(dy, s, weight, dsum, dtype, eps=1e-6):
    dy, s = d(dy), d(s)
    m, n = s.shape
    r = 1 / torch.sqrt((s * s).mean(dim=1, keepdim=True) + eps)
    h, g = s * r, dy if weight is None else dy * d(weight)
    size = r * (g.abs() + h.abs() * (g * h).abs().mean(dim=1, keepdim=True))
    exact, _ = rmsnorm_backward(dy, s, weight, dsum, eps)
    err = size * 160 * U32 + (0 if dsum is None else d(dsum).abs() * 2 * U32)
    return rounded(exact, dtype, err), (dy * h).abs().sum(dim=0) * (m + 160) * U32 + 2.0 ** -126


def linear_bounds(x, w, bias, activation, residual, dtype, x_scale=None, w_scale=None):
    """(bound of z in bf16, bound of out)."""
    z, out = linear(x, w, bias, activation, residual, x_scale, w_scale)
    size, _ = linear(d(x).abs(), d(w).abs(), None, "none", None, x_scale, w_scale)
    k = x.shape[1]
    err = size * (k + 8) * U32 + z.abs() * 8 * U32 + (0 if bias is None else d(bias).abs() * 8 * U32)
    # no activation's slope passes 1.2; its own arithmetic is good to 2^-18 of its argument
    y_err = 1.2 * err + (0 if activation in ("none", "relu") else 2.0 ** -18 * z.abs())
    if residual is not None:
        y_err = y_err + d(residual).abs() * 4 * U32 + out.abs() * 4 * U32
    return rounded(z, torch.bfloat16, err), rounded(out, dtype, y_err)


def activation_backward_bounds(dout, pre, activation):
    """(bound of dpre in bf16, bound of dbias)."""
    do = d(dout)
    exact = do * (torch.ones_like(do) if activation == "none" else act_grad(d(pre), activation))
    err = do.abs() * 2.0 ** -17 if activation not in ("none", "relu") else do.abs() * 0
    m = do.shape[0]
    return rounded(exact, torch.bfloat16, err), err.sum(dim=0) + exact.abs().sum(dim=0) * (m + 64) * U32 + 2.0 ** -126


def product_bound(a, b, dtype, old=None):
    """|a . b| of a (m x k) and b (k x n), plus an old value."""
    exact = d(a) @ d(b)
    size = d(a).abs() @ d(b).abs()
    if old is not None:
        exact, size = exact + d(old), size + d(old).abs()
    return exact, rounded(exact, dtype, size * (a.shape[1] + 8) * U32)
