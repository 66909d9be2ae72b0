"""A pre-norm feed-forward layer out of the layer operators, trained a few steps in bf16 and then served in e4m3.

    python examples/feed_forward.py [--tokens 512] [--hidden 1024] [--inner 4096] [--steps 20]

Training (bf16, fp32 gradients and master weights):

    s, h = norm(x + residual)          layer_rmsnorm
    a    = gelu_tanh(h w1^T + b1)      layer_linear, keeping the pre-activation
    y    = a w2^T + s                  layer_linear, the residual stream in its epilogue

and back through layer_linear_backward, layer_activation_backward and layer_rmsnorm_backward, which joins the stream's own
gradient. Serving: the same layer with both weights quantised once to e4m3 rows; the norm writes the first product's operand
and its row scales itself. Needs an MI355X.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

E4M3_MAX = 448.0


class FeedForward:
    """Weights, gradients and buffers for batches of `tokens` rows."""

    def __init__(self, tokens: int, hidden: int, inner: int, seed: int = 0, eps: float = 1e-6):
        import torch

        import persistent_tiled_gemm_amd as ptg

        self.ptg, self.torch, self.eps = ptg, torch, eps
        self.plan = ptg.layer_create(torch.cuda.current_device())
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def master(rows, cols):
            return torch.randn(rows, cols, generator=g, device="cuda") / math.sqrt(cols)

        # fp32 master weights; the bf16 copies are what the products read
        self.master = {"w1": master(inner, hidden), "w2": master(hidden, inner), "b1": torch.zeros(inner, device="cuda"),
                       "gain": torch.ones(hidden, device="cuda")}
        self.grad = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.refresh()

        def empty(rows, cols):
            return torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")

        self.s, self.h, self.y = empty(tokens, hidden), empty(tokens, hidden), empty(tokens, hidden)
        self.pre, self.a = empty(tokens, inner), empty(tokens, inner)
        self.da, self.dpre = empty(tokens, inner), empty(tokens, inner)
        self.dh, self.dx = empty(tokens, hidden), empty(tokens, hidden)

    def refresh(self):
        self.bf16 = {k: v.to(self.torch.bfloat16) for k, v in self.master.items()}

    def forward(self, x, residual):
        p, w = self.ptg, self.bf16
        p.layer_rmsnorm(x, w["gain"], self.h, residual=residual, sum_out=self.s, eps=self.eps)
        p.layer_linear(self.h, w["w1"], self.a, self.plan, bias=w["b1"], activation="gelu_tanh", pre=self.pre)
        p.layer_linear(self.a, w["w2"], self.y, self.plan, residual=self.s)
        return self.y

    def backward(self, dy):
        """Gradients of the weights into self.grad (added), of x and of the residual as the return value."""
        p, w, g = self.ptg, self.bf16, self.grad
        p.layer_linear_backward(dy, self.a, w["w2"], self.plan, dx=self.da, dw=g["w2"], accumulate=True)
        p.layer_activation_backward(self.da, self.pre, self.dpre, self.plan, activation="gelu_tanh", dbias=g["b1"], accumulate=True)
        p.layer_linear_backward(self.dpre, self.h, w["w1"], self.plan, dx=self.dh, dw=g["w1"], accumulate=True)
        # dy also reaches s past the products: it joins the norm's gradient
        p.layer_rmsnorm_backward(self.dh, self.s, w["gain"], self.dx, g["gain"], self.plan, dsum=dy, accumulate=True, eps=self.eps)
        return self.dx

    def descend(self, rate: float):
        for k, v in self.master.items():
            v -= rate * self.grad[k]
            self.grad[k].zero_()
        self.refresh()


class Served:
    """The layer with e4m3 weights, for one step's tokens."""

    def __init__(self, trained: FeedForward, tokens: int):
        torch = trained.torch
        self.ptg, self.torch, self.plan, self.eps, self.w = trained.ptg, torch, trained.plan, trained.eps, trained.bf16
        self.q = {}
        for name in ("w1", "w2"):  # laid out once
            w = trained.master[name]
            scale = w.abs().amax(dim=1) / E4M3_MAX
            self.q[name] = ((w / scale[:, None]).to(torch.float8_e4m3fn), scale)
        hidden, inner = self.w["w2"].shape
        self.h8 = torch.empty(tokens, hidden, dtype=torch.float8_e4m3fn, device="cuda")
        self.a8 = torch.empty(tokens, inner, dtype=torch.float8_e4m3fn, device="cuda")
        self.h_scale, self.a_scale = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        self.a = torch.empty(tokens, inner, dtype=torch.bfloat16, device="cuda")

    def step(self, x, residual, out):
        """residual += x, in place; out = residual + the layer's output."""
        p, w = self.ptg, self.w
        p.layer_rmsnorm(x, w["gain"], self.h8, residual=residual, sum_out=residual, scale=self.h_scale, eps=self.eps)
        (w1, s1), (w2, s2) = self.q["w1"], self.q["w2"]
        p.layer_linear(self.h8, w1, self.a, self.plan, bias=w["b1"], activation="gelu_tanh", x_scale=self.h_scale, w_scale=s1)
        # the second product's operand: e4m3 rows of the activations
        amax = self.a.float().abs().amax(dim=1)
        self.a_scale.copy_(self.torch.where(amax == 0, self.torch.ones_like(amax), amax / E4M3_MAX))
        self.a8.copy_(self.a.float() / self.a_scale[:, None])
        p.layer_linear(self.a8, w2, out, self.plan, residual=residual, x_scale=self.a_scale, w_scale=s2)
        return out


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args(argv)
    import torch

    layer = FeedForward(a.tokens, a.hidden, a.inner)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, residual, target = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    losses = []
    for _ in range(a.steps):
        diff = layer.forward(x, residual).float() - target.float()
        losses.append(diff.square().mean().item())
        layer.backward((2.0 / a.hidden * diff).to(torch.bfloat16))
        layer.descend(4.0 / a.tokens)
    layer.ptg.layer_sync(layer.plan)
    print(f"training: mean squared error {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps")

    served = Served(layer, 4)
    want = layer.forward(x, residual)[:4].float()
    out = torch.empty(4, a.hidden, dtype=torch.bfloat16, device="cuda")
    got = served.step(x[:4], residual[:4].clone(), out).float()
    layer.ptg.layer_sync(layer.plan)
    off = ((got - want).norm() / want.norm()).item()
    print(f"serving in e4m3: {off:.4f} off the bf16 layer (2-norm, relative)")
    return losses, off


if __name__ == "__main__":
    main()
