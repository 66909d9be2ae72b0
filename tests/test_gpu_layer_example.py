"""The feed-forward example: its gradients against the fp64 chain, its training step and its e4m3 form."""

import pytest
import torch

from examples import feed_forward
from oracle import layer_ref as ref
from tests.layer_util import normal, say

pytestmark = pytest.mark.gpu


def test_gradients_follow_the_chain_rule():
    """Every gradient of the layer against autograd in fp64 of the same formulas. The chain rounds each tensor it hands on
    to bf16 (half a step: 2^-8 of an element); its six roundings in a row, each spread over a whole product's terms, stay
    within 6 2^-8 of the gradient's norm."""
    t, h, f = 72, 136, 264
    layer = feed_forward.FeedForward(t, h, f)
    x, r, dy = normal(1, t, h), normal(2, t, h), normal(3, t, h)
    layer.forward(x, r)
    dx = layer.backward(dy)
    layer.ptg.layer_sync(layer.plan)
    p = {k: ref.d(v).requires_grad_(True) for k, v in layer.bf16.items()}
    xs = ref.d(x).requires_grad_(True)
    s = xs + ref.d(r)
    hid = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + layer.eps) * p["gain"]
    a = ref.act(hid @ p["w1"].t() + p["b1"], "gelu_tanh")
    ((a @ p["w2"].t() + s) * ref.d(dy)).sum().backward()
    for name, got, want in [("x", dx, xs.grad)] + [(k, layer.grad[k], p[k].grad) for k in p]:
        off = ((ref.d(got) - want).norm() / want.norm()).item()
        say(name, off)
        assert off <= 6 * 2.0 ** -8, name


def test_example_trains_and_serves():
    losses, off = feed_forward.main(["--tokens", "96", "--hidden", "256", "--inner", "1024", "--steps", "15"])
    assert losses[-1] < 0.8 * losses[0]
    # two e4m3 products: each operand off by at most 2^-4 of an element, against a residual stream that is exact
    assert off <= 4 * 2.0 ** -4
