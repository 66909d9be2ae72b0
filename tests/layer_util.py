"""Helpers of the layer operators' GPU tests: seeded inputs, guarded outputs and the comparison with a bound."""

from __future__ import annotations

import torch

GUARD = 96.0  # what lies around an output; exact in every type used


def say(*a):
    print(*a, flush=True)


def normal(seed, *shape, scale=1.0, dtype=torch.bfloat16, pad=0):
    """N(0, scale^2) on the GPU, made on the CPU from the seed; with `pad`, a column slice of a wider buffer."""
    t = (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * scale).to(dtype).cuda()
    if not pad:
        return t
    wide = torch.full((shape[0], shape[1] + pad), GUARD, device="cuda").to(dtype)
    wide[:, : shape[1]] = t
    return wide[:, : shape[1]]


class Out:
    """An output inside a larger buffer: rows are at least `pad` elements further apart than they are long (a multiple
    of 16 elements apart, so that the output's first row is 16-byte aligned in every type) and a row lies before and
    after. t is the output; check() finds writes outside it."""

    def __init__(self, m, n, dtype, pad=16, fill=None):
        self.buf = torch.full((m + 2, (n + pad + 15) // 16 * 16), GUARD, device="cuda").to(dtype)
        self.t = self.buf[1: m + 1, :n]
        if fill is not None:
            self.t.copy_(fill)

    def check(self):
        b = self.buf.float().cpu()
        m, n = self.t.shape
        assert (b[0] == GUARD).all() and (b[m + 1] == GUARD).all() and (b[:, n:] == GUARD).all(), "a write outside the output"


def within(got, exact, bound, what):
    got = got.detach().cpu().to(torch.float64)
    off = (got - exact).abs()
    bad = ~(off <= bound)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off; at {i}: got {got[i]}, exact {exact[i]}, "
                             f"bound {bound[i]}; largest off / bound {(off / bound).max()}")
