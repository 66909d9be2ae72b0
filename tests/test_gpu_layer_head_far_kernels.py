"""The calls of head_far_cases.CASES against the fp64 oracle."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from tests import head_far_cases
from tests import test_gpu_layer_i8 as i8_tests
from tests import test_gpu_layer_loss as loss_tests
from tests.layer_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def plan():
    with ptg.layer_create(torch.cuda.current_device()) as p:
        yield p


@pytest.mark.parametrize("what,kind,m,n,k", head_far_cases.CASES)
def test_every_kernel(plan, what, kind, m, n, k):
    say(what, kind, m, n, k)
    if kind == "i8":
        i8_tests.check(plan, m, n, k, torch.bfloat16, "silu")
    else:
        loss_tests.check_sampled(plan, m, n, k, backward=False)
