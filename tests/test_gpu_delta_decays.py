"""dg of det_delta_rule_bwd against float64, relative to itself: gates that forget a state within a token or two, and
tokens that reset a state that is kept otherwise. The gradient of such a gate is smaller than the terms of its
neighbours by its decay, so what these leave of their rounding would be all of it."""
import math

import pytest
import torch

from tests import ref64_delta as R
from tests.test_gpu_delta_rule import BF, F32, X, bwd, fwd, make, to_dev

pytestmark = pytest.mark.gpu


def gates(kind, T, H, gen):
    if kind == "resets":     # kept otherwise: every eleventh token or so forgets, and neighbours do
        g = -0.02 * torch.rand(T, H, generator=gen)
        at = torch.rand(T, H, generator=gen) < 0.09
        return torch.where(at, -8.0 - 32.0 * torch.rand(T, H, generator=gen), g)
    if kind == "mixed":      # any decay next to any other
        return -torch.exp(8.0 * torch.rand(T, H, generator=gen) - 4.0)
    return torch.full((T, H), kind) * (1.0 + 0.1 * torch.rand(T, H, generator=gen))


def limits(dtype, mag, want, chunks, dv):
    """Largest errors, one by one [T, H] and in the norm of all: eight and two standard deviations (see ref64_delta). In
    the norm of all the magnitude is what products over dv channels have, whose signs are random here as are their
    errors': 1 / sqrt(dv) of the bound by norms."""
    sd = R.allowed(chunks) / 8.0 * 2.0 ** -24 * mag
    rounded = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -126
    return 8.0 * sd + rounded, (2.0 / math.sqrt(dv) * sd + rounded).norm().item()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", [-0.5, -5.0, -12.0, -30.0, -80.0, "resets", "mixed"])
@pytest.mark.parametrize("dk,dv,offs", [(64, 64, [0, 150]), (128, 128, [0, 64, 100, 250]), (96, 80, [3, 50, 50, 200]), (33, 128, [0, 31])])
def test_dg_keeps_its_digits(dk, dv, offs, kind, dtype):
    T, H = offs[-1] + 2, 4
    gen = torch.Generator().manual_seed(dk)
    h = make(T, offs, 2, H, dk, dv, dtype, seed=dk + 1)
    h["g"] = gates(kind, T, H, gen)
    o, s1, _, kept = R.delta(*(h[n] for n in X), offs, h["s0"], dk ** -0.5)
    want, _ = R.delta_bwd(h["do"], kept, h["ds1"], 2)
    mag = R.delta_dg_mag(kept, h["do"], h["s0"], h["ds1"])
    d = to_dev(h)
    rows = slice(offs[0], offs[-1])
    got, want, mag = bwd(d, fwd(d))["dg"].cpu().double()[rows], want["dg"][rows], mag[rows]
    each, norm = limits(dtype, mag, want, 4, dv)
    off = (got - want).abs()
    assert off.norm().item() <= norm, "relative to dg's norm %.3g, allowed %.3g" % (off.norm() / want.norm(), norm / want.norm())
    assert (off <= each).all(), "worst %.3g of its limit" % (off / each).max()
