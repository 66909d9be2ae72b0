"""What the cross entropy's gradient promises of a vocabulary that w masks, and of one output beside the other."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import Out, say, within
from tests.test_gpu_layer_loss import forward, head

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def plan():
    with ptg.layer_create(torch.cuda.current_device()) as p:
        yield p


def scratch(m, n, k, pieces=1):
    return torch.empty(ptg.layer_cross_entropy_scratch(m, n, k, pieces), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("m,n,k,pieces", [(4, 520, 64, 1), (40, 1032, 264, 3), (300, 1032, 136, 2), (937, 88, 1024, 1)])
def test_a_vocabulary_masked_in_w(plan, m, n, k, pieces):
    """Entries masked by -infinity have dz = 0: dw is the gradient of the others, zeros for the masked; dx is right except in
    the columns where w is infinite, which are NaN."""
    say("masked vocabulary", m, n, k, pieces)
    x, w, label = head(m, n, k)
    x[:, 0], w[:, 0] = 1.0, 0.0
    kept = torch.ones(n, dtype=torch.bool)
    kept[5], kept[n // 3: n // 2] = False, False
    w[~kept.cuda(), 0] = -float("inf")
    place = torch.cumsum(kept, 0) - 1  # of a kept entry among them
    label = torch.where((label >= 0) & ~kept.cuda()[label.clamp(min=0)], torch.zeros_like(label), label)
    lse = forward(plan, x, w, label)[0][1: m + 1].clone()
    dx, dw = Out(m, k, F32), Out(n, k, F32)
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch(m, n, k, pieces), plan, dx=dx.t, dw=dw.t)
    torch.cuda.synchronize()
    dx.check()
    dw.check()
    few = torch.where(label.cpu() < 0, label.cpu(), place[label.cpu().clamp(min=0)])
    (want_dx, dx_off), (want_dw, dw_off) = ref.cross_entropy_backward_bounds(x, w[kept.cuda()], few, lse, F32, F32)
    assert (dw.t[~kept.cuda()] == 0).all()
    within(dw.t.cpu()[kept], want_dw, dw_off, "dw")
    within(dx.t.cpu()[:, 1:], want_dx[:, 1:], dx_off[:, 1:], "dx")
    assert torch.isnan(dx.t[:, 0]).all()


@pytest.mark.parametrize("m,n,k", [(150, 2056, 264), (777, 10248, 520)])
@pytest.mark.parametrize("dx_t", [BF16, F32])
def test_dw_alone_and_beside_dx(plan, m, n, k, dx_t):
    """One scratch for all three calls. The sum of a bf16 dx takes some of it, so that the pieces may be others and with them
    the order of sums: each result is within the bounds. An fp32 dx takes none: the same pieces, the same bits."""
    say("dw beside dx", m, n, k, dx_t)
    x, w, label = head(m, n, k)
    lse = forward(plan, x, w, label)[0][1: m + 1].clone()
    room = scratch(m, n, k, 2)
    both, alone = (Out(m, k, dx_t), Out(n, k, F32)), (Out(m, k, dx_t), Out(n, k, F32))
    ptg.layer_cross_entropy_backward(x, w, label, lse, room, plan, dx=both[0].t, dw=both[1].t)
    ptg.layer_cross_entropy_backward(x, w, label, lse, room, plan, dx=alone[0].t)
    ptg.layer_cross_entropy_backward(x, w, label, lse, room, plan, dw=alone[1].t)
    torch.cuda.synchronize()
    want = ref.cross_entropy_backward_bounds(x, w, label, lse, dx_t, F32)
    for name, exact, a, b in zip(("dx", "dw"), want, both, alone):
        for t in (a, b):
            t.check()
            within(t.t, *exact, name)
        if dx_t == F32 or name == "dx":
            assert torch.equal(a.t, b.t), name
