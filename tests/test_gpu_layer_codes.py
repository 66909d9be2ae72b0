"""The e4m3 codes of the norm are the fp32 quotient y / scale rounded to nearest: ties and what lies next to them."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from tests.layer_util import normal, say

pytestmark = pytest.mark.gpu

BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


# every row-group size; enough values that some quotients lie next to a tie (about one in a million does)
@pytest.mark.parametrize("m,n,small", [(16384, 512, 1.0), (4096, 2056, 1.0), (2048, 8192, 1.0), (512, 16392, 1.0), (1024, 4104, 2.0 ** -110)])
def test_codes_are_the_quotient_by_the_scale(m, n, small):
    """The same call with fp32 output gives the very y that the codes are made of. `small`: a weight that takes the
    scales far down, where a remainder could fall among the subnormal numbers."""
    say("norm codes", m, n, small)
    x = normal(1, m, n, scale=3.0)
    x[:, ::509] *= 20.0
    w = (1 + 0.2 * normal(2, n, dtype=F32)) * small
    codes, scale = torch.empty(m, n, dtype=E4M3, device="cuda"), torch.empty(m, device="cuda")
    y = torch.empty(m, n, device="cuda")
    ptg.layer_rmsnorm(x, w, codes, scale=scale)
    ptg.layer_rmsnorm(x, w, y)
    torch.cuda.synchronize()
    want = (y.cpu() / scale.cpu()[:, None]).to(E4M3)
    off = want.float() != codes.cpu().float()
    assert not off.any(), f"{int(off.sum())} of {off.numel()} codes are not round(y / scale)"
