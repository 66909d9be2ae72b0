"""Rows whose offsets pass 32 bits: the layer operators on matrices with the largest row stride, against the same call on
matrices without gaps (the same kernels in the same order: equal bits)."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from tests.layer_util import normal

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
STRIDE, M, N, K = 1 << 20, 4160, 256, 128  # the last row starts 8.1 GiB in


@pytest.fixture(scope="module")
def plan():
    with ptg.layer_create(torch.cuda.current_device()) as p:
        yield p


@pytest.fixture(scope="module")
def far():
    """Two far matrices of at least M rows, shared by the tests (bf16, 8.1 GiB each)."""
    buffers = [torch.empty(M * STRIDE, dtype=BF16, device="cuda") for _ in range(2)]
    yield lambda i, m, n: buffers[i].as_strided((m, n), (STRIDE, 1))
    buffers.clear()


def copied(far, i, t):
    f = far(i, *t.shape)
    f.copy_(t)
    return f


def test_norm(far):
    x, g = normal(1, M, N), normal(2, N)
    want, got = torch.empty_like(x), far(1, M, N)
    ptg.layer_rmsnorm(x, g, want)
    ptg.layer_rmsnorm(copied(far, 0, x), g, got)
    assert torch.equal(got, want)


def test_norm_backward(plan, far):
    s, dy, g = normal(1, M, N), normal(2, M, N), normal(3, N)
    want, dg, dg_want = torch.empty_like(s), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    ptg.layer_rmsnorm_backward(dy, s, g, want, dg_want, plan)
    got = far(1, M, N)
    ptg.layer_rmsnorm_backward(dy, copied(far, 0, s), g, got, dg, plan)
    assert torch.equal(got, want) and torch.equal(dg, dg_want)


@pytest.mark.parametrize("m,n", [(M, N), (40, M)])
def test_linear(plan, far, m, n):
    """Far x, residual and out with many rows; far w with few."""
    x, w, r = normal(1, m, K), normal(2, n, K, scale=0.1), normal(3, m, n)
    want = torch.empty_like(r)
    ptg.layer_linear(x, w, want, plan, residual=r, activation="silu")
    if m == M:
        got = torch.empty_like(r)
        ptg.layer_linear(copied(far, 0, x), w, got, plan, residual=copied(far, 1, r), activation="silu")
        assert torch.equal(got, want)
        got = far(0, m, n)
        ptg.layer_linear(x, w, got, plan, residual=r, activation="silu")
    else:
        got = torch.empty_like(r)
        ptg.layer_linear(x, copied(far, 0, w), got, plan, residual=r, activation="silu")
    assert torch.equal(got, want)


def test_activation_backward(plan, far):
    do, pre = normal(1, M, N), normal(2, M, N)
    want, db, db_want = torch.empty_like(do), torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    ptg.layer_activation_backward(do, pre, want, plan, activation="gelu", dbias=db_want)
    got = copied(far, 1, pre)
    ptg.layer_activation_backward(copied(far, 0, do), got, got, plan, activation="gelu", dbias=db)
    assert torch.equal(got, want) and torch.equal(db, db_want)


def test_linear_backward(plan, far):
    dpre, x, w = normal(1, M, N), normal(2, M, K), normal(3, N, K, scale=0.1)
    dx_want, dw_want = torch.empty(M, K, dtype=BF16, device="cuda"), torch.empty(N, K, device="cuda")
    ptg.layer_linear_backward(dpre, x, w, plan, dx=dx_want, dw=dw_want)
    dx, dw = torch.empty_like(dx_want), torch.empty_like(dw_want)
    ptg.layer_linear_backward(copied(far, 0, dpre), copied(far, 1, x), w, plan, dx=dx, dw=dw)
    assert torch.equal(dx, dx_want) and torch.equal(dw, dw_want)
    dx = far(0, M, K)
    ptg.layer_linear_backward(dpre, None, w, plan, dx=dx)
    assert torch.equal(dx, dx_want)
