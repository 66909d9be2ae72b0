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


def rmsnorm_codes_bound(v):
    """Of int8 codes against the unrounded quotients v: half a code, and the quotient's own error. The root is in
    both of its parts and cancels; left are the sum s (in both), two products in each, two divisions: 8 roundings."""
    return 0.5 + 10 * U32 * v.abs()


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


# ---- rows in 8 bits, and the cross entropy of an output head

TOPS = {torch.int8: 127.0, torch.float8_e4m3fn: E4M3_MAX}


def quantise_rows(x, dtype):
    """(scale, codes) of layer_quantize, which defines both by fp32 quotients: IEEE divisions here."""
    x = x.detach().cpu().to(torch.float32)
    top = x.abs().amax(dim=1)
    bad = ~torch.isfinite(x).all(dim=1)
    scale = torch.where(top == 0, torch.ones_like(top), (top / torch.full_like(top, TOPS[dtype])).clamp(min=2.0 ** -126))
    scale[bad] = float("nan")
    q = x / scale[:, None]
    if dtype == torch.int8:
        return scale, torch.where(bad[:, None], torch.zeros_like(q), q.round()).to(torch.int8)
    return scale, q.to(dtype)


def cross_entropy(x, w, label):
    """(lse, loss); a negative label's loss is 0, one past the vocabulary NaN."""
    z = d(x) @ d(w).t()
    label = label.cpu()
    lse = torch.logsumexp(z, dim=1)
    past = label >= z.shape[1]
    at = torch.where(past, torch.zeros_like(label), label).clamp(min=0)
    loss = torch.where(label < 0, torch.zeros_like(lse), lse - z.gather(1, at[:, None])[:, 0])
    return lse, torch.where(past, torch.full_like(loss, float("nan")), loss)


def _logits_error(x, w):
    """How far a logit may be off: an fp32 sum of k products."""
    return (d(x).abs() @ d(w).abs().t()) * (x.shape[1] + 8) * U32


def cross_entropy_bounds(x, w, label):
    """(bound of lse, bound of loss). A row's logits move lse by at most the largest of their errors. A sum of n
    exponentials: chains of 32 in a lane and of n / 16 / 8 blocks in the join, and the trees; 2^-23 and |t| 2^-24 of each
    exponential e^t, |t| e^t below 0.4. lse is the maximum plus a logarithm: a step of each."""
    e = _logits_error(x, w)
    z = d(x) @ d(w).t()
    lse, loss = cross_entropy(x, w, label)
    n = z.shape[1]
    lse_err = e.amax(dim=1) + (n / 128 + 128) * U32 + 4 * U32 * (lse.abs() + z.amax(dim=1).abs())
    at = label.cpu().clamp(min=0, max=n - 1)[:, None]
    loss_err = torch.where(label.cpu() < 0, torch.zeros_like(lse), lse_err + e.gather(1, at)[:, 0] + 2 * U32 * loss.abs())
    return lse_err, loss_err


def logit_grad(x, w, label, lse, weight=None):
    """dz at a given lse."""
    p = torch.exp(d(x) @ d(w).t() - d(lse)[:, None])
    label = label.cpu()
    rows = torch.arange(p.shape[0])[label >= 0]
    p[rows, label[label >= 0]] -= 1.0
    if weight is not None:
        p = p * d(weight)[:, None]
    p[label < 0] = 0.0
    return p


def cross_entropy_backward(x, w, label, lse, weight=None, dloss=None):
    """(dx, dw)."""
    dz = logit_grad(x, w, label, lse, weight) * (1.0 if dloss is None else d(dloss).reshape(()))
    return dz @ d(w), dz.t() @ d(x)


def cross_entropy_backward_bounds(x, w, label, lse, dx_dtype, dw_dtype, weight=None, dloss=None, old=None):
    """(bound of dx, bound of dw). exp(z - lse): its argument is off by the logit's error and by steps of z and lse, the
    exponential by 2^-23; dz is then rounded to bf16 and multiplied in fp32."""
    g = 1.0 if dloss is None else d(dloss).reshape(()).abs()
    z = d(x) @ d(w).t()
    dz = logit_grad(x, w, label, lse, weight)
    size = torch.ones(z.shape[0], dtype=torch.float64) if weight is None else d(weight).abs()
    size = torch.where(label.cpu() < 0, torch.zeros_like(size), size)[:, None]
    t = _logits_error(x, w) + 3 * U32 * (z.abs() + d(lse).abs()[:, None])
    p_err = torch.exp(z - d(lse)[:, None]) * (torch.expm1(t) + 4 * U32) + 2 * U32
    err = size * p_err
    err = err + HALF_STEP[torch.bfloat16] * (dz.abs() + err) + TINY[torch.bfloat16]
    m, n = z.shape
    dx, dw = cross_entropy_backward(x, w, label, lse, weight, dloss)
    dx_err = g * (err @ d(w).abs() + (dz.abs() @ d(w).abs()) * (n + 64) * U32)
    dw_err = g * (err.t() @ d(x).abs() + (dz.t().abs() @ d(x).abs()) * (m + 64) * U32)
    if old is not None:
        dw, dw_err = dw + d(old), dw_err + d(old).abs() * 2 * U32
    return (dx, rounded(dx, dx_dtype, dx_err)), (dw, rounded(dw, dw_dtype, dw_err))
