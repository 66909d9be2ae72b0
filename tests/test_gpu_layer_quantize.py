"""Rows in 8 bits against their definition by fp32 quotients: codes and scales are equal, bit for bit."""

import pytest
import torch

import persistent_tiled_gemm_amd as ptg
from oracle import layer_ref as ref
from tests.layer_util import Out, normal, say, within

pytestmark = pytest.mark.gpu

I8, E4M3, BF16, F32 = torch.int8, torch.float8_e4m3fn, torch.bfloat16, torch.float32


def check(x, dtype, pad=16):
    m, n = x.shape
    out = Out(m, n, dtype, pad)
    scale = torch.full((m + 2,), -7.0, device="cuda")
    ptg.layer_quantize(x, out.t, scale[1: m + 1])
    torch.cuda.synchronize()
    want_scale, want = ref.quantise_rows(x, dtype)
    out.check()
    assert scale[0] == -7.0 and scale[m + 1] == -7.0, "a write outside the scales"
    assert torch.equal(scale[1: m + 1].cpu().nan_to_num(-1.0), want_scale.nan_to_num(-1.0))
    got = out.t.cpu().contiguous().view(torch.uint8)
    off = got != want.view(torch.uint8)
    if dtype == E4M3:
        off &= ~(torch.isnan(out.t.cpu().float()) & torch.isnan(want.float()))
    assert not off.any(), f"{int(off.sum())} of {off.numel()} codes, the first at {tuple(off.nonzero()[0].tolist())}"


# every row group's size, one row to more rows than there are groups, and rows that are read twice
SHAPES = [(1, 8), (3, 512), (5, 520), (1000, 64), (9, 1024), (7, 1032), (1, 2048), (33, 2056), (2, 4096), (3, 4104), (1, 8192), (65, 8200),
          (2, 16384), (3, 16392), (1, 32768), (2, 32776), (3, 65536), (5000, 264), (2500, 1544), (700, 9000)]


@pytest.mark.parametrize("m,n", SHAPES)
@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("t", [BF16, F32])
def test_codes_and_scales(m, n, dtype, t):
    say("quantize", m, n, dtype, t)
    x = normal(m + n, m, n, dtype=t, pad=8)
    x[:, :: 509] *= 20.0
    check(x, dtype)


@pytest.mark.parametrize("dtype", [I8, E4M3])
def test_ties_and_borders(dtype):
    """Quotients at and next to the half-way points between codes, where a quotient that is off by one step shows."""
    rows = []
    for top in (127.0, 254.0, 1.0, 0.3, 3e-6, 1e30, 448.0, 0.875):
        scale = torch.tensor(top) / torch.tensor(ref.TOPS[dtype])
        half = (torch.arange(-126, 126) + 0.5) * scale
        x = torch.cat([torch.tensor([top]), half, torch.nextafter(half, torch.tensor(1e38)), torch.nextafter(half, torch.tensor(-1e38))])
        rows.append(torch.cat([x, torch.zeros(768 - len(x))]))
    check(torch.stack(rows).cuda(), dtype)


@pytest.mark.parametrize("dtype", [I8, E4M3])
@pytest.mark.parametrize("t", [BF16, F32])
@pytest.mark.parametrize("n", [64, 1544, 40000])
def test_empty_tiny_huge_and_non_finite_rows(dtype, t, n):
    x = normal(3, 12, n, dtype=F32)
    x[1] = 0.0
    x[2] *= 1e-38
    x[3] *= 1e-42
    x[4] = 0.0
    x[4, 5] = -1e-45
    x[5] *= 3e37
    x[6, 7] = float("inf")
    x[7, n - 1] = -float("inf")
    x[8, 3] = float("nan")
    x[9] = -0.0
    x[10] = 2.5
    check(x.to(t), dtype)


def check_norm(x, residual=None, weight=None, sum_out=False):
    m, n = x.shape
    out, scale = Out(m, n, I8), torch.full((m,), -1.0, device="cuda")
    kept = Out(m, n, x.dtype) if sum_out else None
    ptg.layer_rmsnorm(x, weight, out.t, residual=residual, sum_out=kept.t if sum_out else None, scale=scale)
    torch.cuda.synchronize()
    out.check()
    s, y = ref.rmsnorm(x, weight, residual)
    top = y.abs().amax(dim=1)
    want = torch.where(top == 0, torch.ones_like(top), (top / 127).clamp(min=2.0 ** -126))
    within(scale, want, want * 100 * ref.U32, "scale")
    v = y / want[:, None]
    within(out.t.float(), v, ref.rmsnorm_codes_bound(v), "codes")
    assert ((out.t.int().abs().amax(dim=1) == 127) | (scale == 1)).all()
    if sum_out:
        within(kept.t, s, ref.rounded(s, x.dtype, s.abs() * 2 * ref.U32), "sum")
        kept.check()


# the norm's row groups: their sizes change at n = 2048 and 8192, chunks per thread in between
@pytest.mark.parametrize("m,n", [(1, 8), (3, 64), (5, 512), (7, 520), (4, 2048), (9, 2056), (2, 4096), (3, 5000), (1, 8192), (6, 8200), (2, 16384),
                                 (2, 32768), (700, 1032)])
@pytest.mark.parametrize("t", [BF16, F32])
def test_norm_to_int8(m, n, t):
    say("norm to int8", m, n, t)
    w = (1 + 0.2 * normal(3, n, dtype=F32)).to(BF16)
    check_norm(normal(1, m, n, scale=3.0, dtype=t, pad=8), normal(2, m, n, dtype=t), w, True)
    check_norm(normal(1, m, n, scale=1e-3, dtype=t))


def test_norm_to_int8_of_zeros_and_non_finite_rows():
    x = normal(1, 5, 264, dtype=F32)
    x[1] = 0.0
    x[2, 7] = float("nan")
    x[3, 8] = float("inf")
    out, scale = torch.empty(5, 264, dtype=I8, device="cuda"), torch.empty(5, device="cuda")
    ptg.layer_rmsnorm(x, None, out, scale=scale)
    torch.cuda.synchronize()
    assert scale[1] == 1.0 and torch.isnan(scale[2:4]).all() and torch.isfinite(scale[[0, 1, 4]]).all()
    assert (out[1:4] == 0).all() and (out[[0, 4]].int().abs().amax(dim=1) == 127).all()


def test_norm_to_int8_refuses():
    x, out = normal(1, 4, 64), torch.empty(4, 64, dtype=I8, device="cuda")
    with pytest.raises(ptg.PtgError) as e:
        ptg.layer_rmsnorm(x, None, out)  # no scale
    assert e.value.status == -1
    with pytest.raises(ptg.PtgError) as e:
        ptg.layer_rmsnorm(x, None, torch.empty_like(x), scale=torch.empty(4, device="cuda"))
    assert e.value.status == -1


def test_nothing_writes_nothing():
    scale = torch.full((4,), -7.0, device="cuda")
    ptg.layer_quantize(torch.empty(0, 64, device="cuda"), torch.empty(0, 64, dtype=I8, device="cuda"), scale[:0])
    ptg.layer_quantize(torch.empty(4, 0, device="cuda"), torch.empty(4, 0, dtype=I8, device="cuda"), scale)
    torch.cuda.synchronize()
    assert (scale == -7.0).all()


def test_refusals():
    x, out, scale = normal(1, 4, 64), torch.empty(4, 64, dtype=I8, device="cuda"), torch.empty(4, device="cuda")
    for args in ((x.half(), out, scale), (x, out.to(BF16), scale), (x, out[:, :56], scale), (x, out, scale[:3]), (x, out, scale.double()),
                 (x, out.t(), scale), (x[0], out, scale), (x, out.cpu(), scale)):
        with pytest.raises(ValueError):
            ptg.layer_quantize(*args)
    for args in ((x[:, :60].contiguous(), out[:, :60].contiguous(), scale), (torch.zeros(4, 68, device="cuda")[:, :60], out[:, :60], scale)):
        with pytest.raises(ptg.PtgError) as e:
            ptg.layer_quantize(*args)
        assert e.value.status == -2
    with pytest.raises(ptg.PtgError) as e:
        ptg.layer_quantize(torch.zeros(4 * 64 + 8, dtype=BF16, device="cuda")[1:257].view(4, 64), out, scale)
    assert e.value.status == -1
