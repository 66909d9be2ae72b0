"""Rows whose offsets pass 32 bits: the quantiser, the int8 product, the cross entropy and its gradient on matrices with the
largest row stride, against the same call on matrices without gaps (the same kernels in the same order: equal bits), and a dz of
more than 4 GiB."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from tests import test_gpu_layer_loss as loss_tests
from tests.layer_util import normal, say

pytestmark = pytest.mark.gpu

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8
STRIDE, M, K = 1 << 20, 4160, 128  # the last row starts 4.1 GiB in with one byte an element


@pytest.fixture(scope="module")
def plan():
    with ptg.layer_create(torch.cuda.current_device()) as p:
        yield p


@pytest.fixture(scope="module")
def far():
    """Two far matrices of M rows (8.1 GiB each), viewed in any type of up to two bytes, or M / 2 rows in four."""
    buffers = [torch.empty(M * STRIDE, dtype=BF16, device="cuda") for _ in range(2)]
    yield lambda i, m, n, t: buffers[i].view(t).as_strided((m, n), (STRIDE, 1))
    buffers.clear()


def copied(far, i, t):
    f = far(i, *t.shape, t.dtype)
    f.copy_(t)
    return f


def codes(seed, m, k):
    return torch.randint(-127, 128, (m, k), generator=torch.Generator().manual_seed(seed)).to(I8).cuda()


@pytest.mark.parametrize("t,m", [(BF16, M), (F32, M // 2)])
def test_quantize(far, t, m):
    x = normal(1, m, 264, dtype=t)
    want, scale, got_scale = torch.empty(m, 264, dtype=I8, device="cuda"), torch.empty(m, device="cuda"), torch.empty(m, device="cuda")
    ptg.layer_quantize(x, want, scale)
    got = far(1, m, 264, I8)
    ptg.layer_quantize(copied(far, 0, x), got, got_scale)
    assert torch.equal(got, want) and torch.equal(got_scale, scale)
    ptg.layer_rmsnorm(x, None, want, scale=scale)
    ptg.layer_rmsnorm(copied(far, 0, x), None, got, scale=got_scale)
    assert torch.equal(got, want) and torch.equal(got_scale, scale)


@pytest.mark.parametrize("m,n,k", [(M, 264, K), (40, M, K), (24, M, 8192)])
def test_int8_linear(plan, far, m, n, k):
    """Far x and residual with many rows; far w with few, read into registers and with x in LDS."""
    say("far int8", m, n, k)
    x, w, r = codes(1, m, k), codes(2, n, k), normal(3, m, n)
    want, got = torch.empty_like(r), torch.empty_like(r)
    ptg.layer_linear(x, w, want, plan, residual=r)
    if m == M:
        ptg.layer_linear(copied(far, 0, x), w, got, plan, residual=copied(far, 1, r))
        assert torch.equal(got, want)
        got = far(0, m, n, BF16)
        ptg.layer_linear(x, w, got, plan, residual=r)
    else:
        ptg.layer_linear(x, copied(far, 0, w), got, plan, residual=r)
    assert torch.equal(got, want)


@pytest.mark.parametrize("m,n,k", [(M, 264, K), (200, M, K), (3, M, K), (24, M, 8192)])
def test_cross_entropy(plan, far, m, n, k):
    say("far loss", m, n, k)
    x, w, label = loss_tests.head(m, n, k)
    lse, loss, far_lse, far_loss = (torch.empty(m, device="cuda") for _ in range(4))
    ptg.layer_cross_entropy(x, w, label, lse, plan, loss=loss)
    if m == M:
        x = copied(far, 0, x)
    else:
        w = copied(far, 0, w)
    ptg.layer_cross_entropy(x, w, label, far_lse, plan, loss=far_loss)
    assert torch.equal(far_lse, lse) and torch.equal(far_loss, loss)


@pytest.mark.parametrize("m,n", [(M, 264), (200, M)])
def test_cross_entropy_backward(plan, far, m, n):
    x, w, label = loss_tests.head(m, n, K)
    lse = torch.empty(m, device="cuda")
    ptg.layer_cross_entropy(x, w, label, lse, plan)
    scratch = torch.empty(ptg.layer_cross_entropy_scratch(m, n, K, 2), dtype=torch.uint8, device="cuda")
    dx, dw = torch.empty(m, K, dtype=BF16, device="cuda"), torch.empty(n, K, dtype=BF16, device="cuda")
    ptg.layer_cross_entropy_backward(x, w, label, lse, scratch, plan, dx=dx, dw=dw)
    big = far(1, max(m, n), K, BF16)
    if m == M:
        far_x, far_w, far_dx, far_dw = copied(far, 0, x), w, big, torch.empty_like(dw)
    else:
        far_x, far_w, far_dx, far_dw = x, copied(far, 0, w), torch.empty_like(dx), big
    ptg.layer_cross_entropy_backward(far_x, far_w, label, lse, scratch, plan, dx=far_dx, dw=far_dw)
    assert torch.equal(far_dx, dx) and torch.equal(far_dw, dw)


def test_a_gradient_of_logits_past_4_gib(plan):
    """One piece over the widest vocabulary: dz has rows of 2 MiB, 4.1 GiB in all."""
    loss_tests.check_sampled(plan, 2080, (1 << 20) - 3, 8)
