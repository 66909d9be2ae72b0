"""The output head's example: its gradients against the fp64 chain and against differences, its training step, its int8 form,
and the operators one after another, in place and replayed from a graph, as a step of serving runs them."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from examples import feed_forward, output_head
from oracle import layer_ref as ref
from tests.layer_util import normal, say

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def chain(model, p, xs, r, label):
    """The model's mean loss in 64 bits."""
    s = xs + ref.d(r)
    hid = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + model.eps) * p["gain"]
    y = ref.act(hid @ p["w1"].t() + p["b1"], "gelu_tanh") @ p["w2"].t() + s
    z = y / torch.sqrt((y * y).mean(dim=1, keepdim=True) + model.eps) * p["last"] @ p["head"].t()
    label = label.cpu()
    kept = label >= 0
    each = torch.logsumexp(z, dim=1) - z.gather(1, label.clamp(min=0)[:, None])[:, 0]
    return each[kept].sum() / max(1, int(kept.sum()))


@pytest.mark.parametrize("pieces", [1, 3])
def test_gradients_follow_the_chain_rule(pieces):
    """Every gradient against autograd in fp64 of the same formulas. The chain rounds each tensor it hands on to bf16 (half a
    step: 2^-8 of an element): h, pre, a, y, the last norm's output, dz, its product, dy and the layer's three before the
    longest path's end, 11 in a row, each spread over a whole product's terms: within 11 2^-8 of the gradient's norm. The
    loss: its logits are off by the four forward roundings of y's and the norm's rows, 4 2^-8 of a logit of size 1 in a mean of 63."""
    t, h, f, v = 72, 136, 264, 776
    model = output_head.Model(t, h, f, v, pieces)
    assert model.scratch.numel() < (2 * t * 1024 if pieces == 1 else 2 * t * 776 + 4 * t * h)
    x, r = normal(1, t, h), normal(2, t, h)
    label = torch.randint(0, v, (t,), device="cuda")
    label[::8] = -1
    got_loss = model.loss(x, r, label).item()
    dx = model.loss_backward(label)
    model.ptg.layer_sync(model.plan)
    p = {k: ref.d(w).requires_grad_(True) for k, w in model.bf16.items()}
    xs = ref.d(x).requires_grad_(True)
    want_loss = chain(model, p, xs, r, label)
    want_loss.backward()
    say("loss", got_loss, want_loss.item())
    assert abs(got_loss - want_loss.item()) <= 4 * 2.0 ** -8
    for name, got, want in [("x", dx, xs.grad)] + [(k, model.grad[k], p[k].grad) for k in p]:
        off = ((ref.d(got) - want).norm() / want.norm()).item()
        say(name, off)
        assert off <= 11 * 2.0 ** -8, name


def test_gradient_of_the_head_against_differences():
    """The loss along a direction of the head's weights, in 64 bits: its central difference is the gradient's product with the
    direction, up to the gradient's own error (11 2^-8 of its norm times the direction's)."""
    t, h, f, v = 24, 64, 128, 520
    model = output_head.Model(t, h, f, v, 2)
    x, r = normal(1, t, h), normal(2, t, h)
    label = torch.randint(0, v, (t,), device="cuda")
    model.loss(x, r, label)
    model.loss_backward(label)
    model.ptg.layer_sync(model.plan)
    p = {k: ref.d(w) for k, w in model.bf16.items()}
    way = ref.d(model.grad["head"])
    step = 1e-4 / way.norm()
    ends = [chain(model, {**p, "head": p["head"] + s * way}, ref.d(x), r, label) for s in (step, -step)]
    slope = ((ends[0] - ends[1]) / (2 * step)).item()
    say("slope", slope, way.square().sum().item())
    assert abs(slope - way.square().sum().item()) <= 11 * 2.0 ** -8 * way.square().sum().item()


def test_example_runs():
    losses, off = output_head.main(["--tokens", "64", "--hidden", "256", "--inner", "512", "--vocab", "1000", "--steps", "3", "--pieces", "2"])
    assert len(losses) == 3 and all(0 < v < 100 for v in losses)
    # three int8 products: each operand's element is off by at most half a code, 2^-8 of its row's largest, which is
    # within 8 times the row's root mean square for rows of a few hundred normal values: 2^-5 of a row's norm an operand
    assert off <= 6 * 2.0 ** -5


def test_feed_forward_serves_in_int8():
    _, off = feed_forward.main(["--tokens", "96", "--hidden", "256", "--inner", "1024", "--steps", "2", "--serve", "int8"])
    assert off <= 4 * 2.0 ** -5  # two products, as above


def test_a_step_of_serving_replays():
    """Norm to int8, product, quantise, product, norm, product in one graph: every replay gives the eager step's bits, with
    the plan's other work between the replays and the stream updated in place each time."""
    model = output_head.Model(8, 256, 1024, 2056)
    served = output_head.Served(model, 8)
    x, residual = normal(3, 8, 256), normal(4, 8, 256)
    want, stream = [], residual.clone()
    for _ in range(4):
        want.append((served.next(x, stream).clone(), stream.clone()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stream = residual.clone()
    with torch.cuda.stream(side):
        served.next(x, residual.clone())
        side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        served.next(x, stream)
    stream.copy_(residual)
    torch.cuda.synchronize()
    for logits, after in want:
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(served.logits, logits) and torch.equal(stream, after)
        model.loss(x, residual, torch.arange(8, device="cuda"))  # the same plan, on another stream, between replays
        torch.cuda.synchronize()
    ptg.layer_sync(model.plan)
