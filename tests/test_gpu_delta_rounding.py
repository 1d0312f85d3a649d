"""A bf16 call of the delta rule computes in float32 and rounds once: of its bf16 outputs no more are another bf16 value
than the rounded float64 result than errors of float32 move over a border between two of them.

An output with the error e goes over a border with probability |e| / step. e is taken from a float32 call of the same
values (whose own tests hold it to float64). A bf16 call's chunks are twice as long, so its errors may be sqrt(2) times
as large, and their sizes spread: three times the expected number is allowed, with four standard deviations of it."""
import math

import pytest
import torch

from tests import ref64_delta as R
from tests.test_gpu_delta_rule import BF, X, bwd, fwd, make, to_dev

pytestmark = pytest.mark.gpu


def moved(got, got32, want, what):
    there = ~torch.isnan(want)
    got, got32, want = got.cpu()[there], got32.cpu().double()[there], want[there]
    step = torch.exp2(torch.floor(torch.log2(want.abs().clamp(min=2.0 ** -126))) - 7)   # of bf16 there
    expected = 3.0 * ((got32 - want).abs() / step).clamp(max=1.0).sum().item()
    count = (got != want.to(BF)).sum().item()
    assert count <= expected + 4.0 * math.sqrt(expected) + 2.0, "%s: %d of %d are not the rounded value, %.1f allowed on average" % (
        what, count, got.numel(), expected)


@pytest.mark.parametrize("g_scale", [0.05, 1.0, 8.0])
@pytest.mark.parametrize("Hk,H,dk,dv,offs", [(2, 4, 128, 128, [0, 300]), (4, 4, 64, 64, [0, 100, 130, 400]), (1, 4, 128, 64, [0, 256]),
                                             (6, 6, 64, 128, list(range(0, 480, 32))), (2, 2, 100, 90, [3, 200])])
def test_outputs_are_rounded_once(Hk, H, dk, dv, offs, g_scale):
    h = make(offs[-1], offs, Hk, H, dk, dv, BF, seed=H + dk, g_scale=g_scale)
    d = to_dev(h)
    e = {n: x.float() if torch.is_tensor(x) and x.dtype == BF else x for n, x in d.items()}
    o, s1, _, kept = R.delta(*(h[n] for n in X), offs, h["s0"], dk ** -0.5)
    moved(fwd(d)["o"], fwd(e)["o"], o, "o")
    # and its gradients
    want, _ = R.delta_bwd(h["do"], kept, h["ds1"], H // Hk)
    r, r32 = bwd(d, fwd(d)), bwd(e, fwd(e))
    for name in ("dv", "dq", "dk", "dbeta", "dg"):
        moved(r[name], r32[name], want[name], name)
