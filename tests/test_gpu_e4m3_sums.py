"""Why e4m3 operands are widened to bf16: the e4m3 matrix instructions drop small products beside large ones, in every form,
and the operators, whose sums are held in 32 bits, do not."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from tests.layer_util import say

pytestmark = pytest.mark.gpu

FORMS = {0: 32, 1: 16, 2: 128, 3: 64}  # terms of one instruction


def cancelling(p):
    """Products 2^p, -2^p and 1."""
    h = p // 2
    return [2.0 ** h, -(2.0 ** h), 1.0], [2.0 ** (p - h), 2.0 ** (p - h), 1.0]


@pytest.mark.parametrize("form", FORMS)
def test_the_instruction_drops_what_lies_far_below_the_largest(form):
    say("e4m3 instruction", form)
    assert ptg.gemm_e4m3_probe([1.0] * FORMS[form], [0.5] * FORMS[form], form) == FORMS[form] / 2  # every term counts
    assert ptg.gemm_e4m3_probe(*cancelling(8), form) == 1.0
    assert ptg.gemm_e4m3_probe(*cancelling(14), form) == 0.0
    with pytest.raises(ptg.PtgError):
        ptg.gemm_e4m3_probe([1.0] * (FORMS[form] + 1), [1.0] * (FORMS[form] + 1), form)


@pytest.mark.parametrize("m", [1, 24, 300])
@pytest.mark.parametrize("p", [8, 14, 16])
def test_the_product_keeps_it(m, p):
    x, w = torch.zeros(m, 64), torch.zeros(264, 64)
    a, b = cancelling(p)
    x[:, :3], w[:, :3] = torch.tensor(a), torch.tensor(b)
    out = torch.empty(m, 264, device="cuda")
    with ptg.layer_create() as plan:
        ptg.layer_linear(x.to(torch.float8_e4m3fn).cuda(), w.to(torch.float8_e4m3fn).cuda(), out, plan)
        torch.cuda.synchronize()
    assert (out == 1.0).all()
