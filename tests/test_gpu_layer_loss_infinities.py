"""The cross entropy where logits are infinite: lse and loss are what the definition gives whichever kernel the sizes pick, and
the other rows are as they were."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import normal, say, within

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
INF = float("inf")

# few rows, k in one share and several; x in LDS, with shares of k that are whole turns of a wave's loads and shares that end inside
# one; tiles, whole and split
PATHS = [(4, 520, 64), (16, 264, 2056), (24, 72, 1008), (36, 136, 72), (11, 4736, 7808), (14, 16328, 2144), (8, 33032, 1288), (2, 20872, 3336),
         (19, 9200, 2056), (32, 3136, 5376), (17, 16720, 4208), (42, 17280, 1032), (64, 3144, 5392), (86, 64, 104), (74, 88, 504), (300, 1032, 136),
         (212, 8200, 640)]


@pytest.fixture(scope="module")
def plan():
    with ptg.layer_create(torch.cuda.current_device()) as p:
        yield p


def check(plan, x, w, label, what):
    m = x.shape[0]
    lse, loss = torch.full((m,), -7.0, device="cuda"), torch.full((m,), -7.0, device="cuda")
    ptg.layer_cross_entropy(x, w, label, lse, plan, loss=loss)
    torch.cuda.synchronize()
    exact = ref.cross_entropy(x, w, label)
    # bounds of the finite rows (an infinity would make its row's, and w's every row's, infinite)
    flat = [torch.where(torch.isfinite(t), t, torch.zeros_like(t)) for t in (x, w)]
    bounds = ref.cross_entropy_bounds(*flat, label)
    for got, want, bound, name in zip((lse, loss), exact, bounds, ("lse", "loss")):
        got, finite = got.cpu().double(), torch.isfinite(want)
        assert torch.equal(got[~finite].nan_to_num(nan=1.0, posinf=2.0, neginf=3.0), want[~finite].nan_to_num(nan=1.0, posinf=2.0, neginf=3.0)), \
            f"{what}: {name} {got[~finite][:8]}, exact {want[~finite][:8]}"
        within(got[finite], want[finite], bound[finite], f"{what}: {name}")
    return exact


@pytest.mark.parametrize("m,n,k", PATHS)
def test_an_infinity_in_x(plan, m, n, k):
    """One infinity a row, at places spread over k, against a column of w with no zero in it: the row's logits are infinite, all
    of one sign or the label's of the other."""
    say("an infinity in x", m, n, k)
    x, w = normal(1, m, k), normal(2, n, k, scale=2.0 / k ** 0.5)
    label = torch.randint(0, n, (m,), generator=torch.Generator().manual_seed(3)).cuda()
    for first in (0, k // 16):
        y, v, t = x.clone(), w.clone(), label.clone()
        rows = [r for r in range(m) if r % 3 != 1][:12]  # the others stay finite
        for i, r in enumerate(rows):
            at = (first + i * (k // len(rows))) % k
            y[r, at] = INF
            v[:, at] = -1.0
            if i % 4 == 1:
                y[r, at] = -INF  # all logits +infinity
            elif i % 4 == 2:
                v[t[r], at] = 1.0  # the label's alone is +infinity
            elif i % 4 == 3:
                v[(t[r] + 1) % n, at] = 1.0  # another one's is
        exact = check(plan, y, v, t, f"{m} {n} {k} from {first}")
        assert not torch.isfinite(exact[0][rows]).any() and torch.isfinite(exact[0][[r for r in range(m) if r % 3 == 1]]).all()


@pytest.mark.parametrize("m,n,k", PATHS)
def test_an_infinite_logit_takes_all(plan, m, n, k):
    """Entries of the vocabulary with an infinite weight: +infinity for the rows that it meets with a positive value, -infinity for
    the others; two in one block of columns and one far from them."""
    say("an infinite logit", m, n, k)
    x, w = normal(1, m, k), normal(2, n, k, scale=2.0 / k ** 0.5)
    label = torch.randint(0, n, (m,), generator=torch.Generator().manual_seed(3)).cuda()
    x[:, 0] = torch.where(torch.arange(m, device="cuda") % 4 < 2, 1.0, -1.0).to(BF16)
    x[:, k - 1] = torch.where(torch.arange(m, device="cuda") % 4 == 1, 1.0, -1.0).to(BF16)
    w[:, 0], w[:, k - 1] = 0.5, -0.25
    w[5, 0], w[9, 0], w[n - 1, k - 1] = INF, INF, INF
    label[0], label[m // 2], label[m - 1] = 5, 9, n - 1
    exact = check(plan, x, w, label, f"{m} {n} {k}")
    rows = torch.arange(m) % 4
    assert (exact[0][rows < 2] == INF).all() and torch.isfinite(exact[0][rows >= 2]).all()
