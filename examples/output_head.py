"""A token predictor's last part: a feed-forward layer, the final norm and the output head, trained on a cross entropy whose
logits are never kept, then served in int8 one token at a time.

    python examples/output_head.py [--tokens 512] [--hidden 512] [--inner 2048] [--vocab 8192] [--steps 20] [--pieces 4]

Training (bf16, fp32 gradients and master weights): feed_forward.FeedForward, then

    h    = norm(y)                     layer_rmsnorm
    loss = mean cross entropy(h w^T)   layer_cross_entropy

and back through layer_cross_entropy_backward, which takes the vocabulary in pieces through a scratch of the given size, and
layer_rmsnorm_backward. Rows with a negative label (padding) are not counted. Serving: the feed-forward layer's int8 form, the
final norm writing int8 rows with their scales (layer_rmsnorm), and the head's logits from the int8 product (layer_linear)
with weights that layer_quantize laid out once; one step is captured into a graph and replayed. Needs an MI355X.
"""

from __future__ import annotations

import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from examples import feed_forward


class Model(feed_forward.FeedForward):
    """The feed-forward layer with a norm and an output head of `vocab` entries behind it."""

    def __init__(self, tokens: int, hidden: int, inner: int, vocab: int, pieces: int = 1, seed: int = 0, eps: float = 1e-6):
        super().__init__(tokens, hidden, inner, seed, eps)
        torch = self.torch
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1)
        more = {"head": torch.randn(vocab, hidden, generator=g, device="cuda") / math.sqrt(hidden), "last": torch.ones(hidden, device="cuda")}
        self.master.update(more)
        self.grad.update({k: torch.zeros_like(v) for k, v in more.items()})
        self.refresh()
        self.top, self.dtop, self.dy = (torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda") for _ in range(3))
        self.lse, self.each = torch.empty(tokens, device="cuda"), torch.empty(tokens, device="cuda")
        size = self.ptg.layer_cross_entropy_scratch(tokens, vocab, hidden, pieces)
        self.scratch = torch.empty(size, dtype=torch.uint8, device="cuda")

    def loss(self, x, residual, label):
        """The mean loss of the rows with a label, on the device."""
        p, w = self.ptg, self.bf16
        y = self.forward(x, residual)
        p.layer_rmsnorm(y, w["last"], self.top, eps=self.eps)
        p.layer_cross_entropy(self.top, w["head"], label, self.lse, self.plan, loss=self.each)
        self.share = 1.0 / (label >= 0).sum().clamp(min=1).float()
        return self.each.sum() * self.share

    def loss_backward(self, label):
        """Gradients of the mean loss into self.grad (added), of x and of the residual as the return value."""
        p, w, g = self.ptg, self.bf16, self.grad
        p.layer_cross_entropy_backward(self.top, w["head"], label, self.lse, self.scratch, self.plan, dx=self.dtop, dw=g["head"],
                                       dloss=self.share, accumulate=True)
        p.layer_rmsnorm_backward(self.dtop, self.y, w["last"], self.dy, g["last"], self.plan, accumulate=True, eps=self.eps)
        return self.backward(self.dy)


class Served(feed_forward.Served):
    """The model in int8, for one step's tokens."""

    def __init__(self, trained: Model, tokens: int):
        torch = trained.torch
        super().__init__(trained, tokens, torch.int8)
        head = trained.master["head"]
        vocab, hidden = head.shape
        self.head, self.head_scale = torch.empty_like(head, dtype=torch.int8), torch.empty(vocab, device="cuda")
        self.ptg.layer_quantize(head, self.head, self.head_scale)
        self.y = torch.empty(tokens, hidden, dtype=torch.bfloat16, device="cuda")
        self.top = torch.empty(tokens, hidden, dtype=torch.int8, device="cuda")
        self.top_scale = torch.empty(tokens, device="cuda")
        self.logits = torch.empty(tokens, vocab, device="cuda")

    def next(self, x, residual):
        """residual += x, in place; the logits (fp32) of the tokens' next ones."""
        self.step(x, residual, self.y)
        self.ptg.layer_rmsnorm(self.y, self.w["last"], self.top, scale=self.top_scale, eps=self.eps)
        self.ptg.layer_linear(self.top, self.head, self.logits, self.plan, x_scale=self.top_scale, w_scale=self.head_scale)
        return self.logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--inner", type=int, default=2048)
    ap.add_argument("--vocab", type=int, default=8192)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--pieces", type=int, default=4)
    a = ap.parse_args(argv)
    import torch

    model = Model(a.tokens, a.hidden, a.inner, a.vocab, a.pieces)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    x, residual = (torch.randn(a.tokens, a.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    label = torch.randint(0, a.vocab, (a.tokens,), generator=g, device="cuda")
    label[-a.tokens // 8:] = -1  # padding
    losses = []
    for _ in range(a.steps):
        losses.append(model.loss(x, residual, label).item())
        model.loss_backward(label)
        model.descend(2.0)
    model.ptg.layer_sync(model.plan)
    print(f"training: cross entropy {losses[0]:.4f} -> {losses[-1]:.4f} in {a.steps} steps (log of {a.vocab}: {math.log(a.vocab):.4f}), "
          f"{model.scratch.numel() / 1e6:.1f} MB of scratch where the logits' gradient takes {2e-6 * a.tokens * a.vocab:.1f}")

    # one step's tokens in int8, beside the bf16 model's logits
    tokens = min(4, a.tokens)
    served = Served(model, tokens)
    model.loss(x, residual, label)
    want = model.top[:tokens].float() @ model.bf16["head"].float().t()
    x_in, stream_in = x[:tokens].clone(), residual[:tokens].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        served.next(x_in, stream_in)  # the plan's last call before a capture is on the capture's stream
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        served.next(x_in, stream_in)
    stream_in.copy_(residual[:tokens])
    graph.replay()
    torch.cuda.synchronize()
    off = ((served.logits - want).norm() / want.norm()).item()
    print(f"serving in int8: logits {off:.4f} off the bf16 model's (2-norm, relative)")
    return losses, off


if __name__ == "__main__":
    main()
