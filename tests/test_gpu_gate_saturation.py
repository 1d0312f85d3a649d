"""The gate's gradient of det_block_norm_bwd where the gate is nearly open or nearly
shut: 1 - sigmoid(gate) keeps its digits, so the tolerances carry that factor."""
import pytest
import torch

from tests import ref64
from tests.test_gpu_block_norm import BF, COL, F32, ROW, bwd, dev, fwd, make

pytestmark = pytest.mark.gpu


def check(T, D, dtype, gate, parts, seed):
    h = make(T, D, dtype, gate=gate, post=parts, alpha=parts, pre=parts, seed=seed)
    # gates from -40 to 80: 1 - sigmoid falls to 2e-35
    g = torch.linspace(-40.0, 80.0, h["gate"].numel()).view_as(h["gate"]).to(dtype)
    h["gate"] = g
    d = dev(h)
    o = fwd(d)
    r = bwd(d, o)
    rs = {k: None if o[k] is None else o[k].cpu() for k in ("rstd_post", "rstd_pre")}
    w = ref64.norm_bwd(h["dy"], h["dh"], h["x"], h["f"], h["gate"], h["w_post"], h["alpha"], h["w_pre"],
                       rs["rstd_post"], rs["rstd_pre"])
    closed = torch.sigmoid(-g.double())
    # dgate = dn n (1 - s) with s = sigmoid(gate): ref64's own form loses the factor's digits above 30, and its magnitude
    # leaves the factor out
    s = torch.sigmoid(g.double())
    want = w["dgate"] / torch.where(s == 1, torch.ones_like(s), 1 - s)
    exact = want * closed
    ok = g.double() < 15                        # above, 1 - s has too few digits in float64 to divide by (2^-53 / 2^-21)
    mag = w["dgate_mag"] * closed
    # roundings: the row sums', and the exponential's argument (|gate| + 3)
    n = 3 * ROW + 60
    got = r["dgate"].cpu().double()
    tol = (n + g.double().abs() + 3) * ref64.U * mag + ref64.HALF_STEP[dtype] * exact.abs() + ref64.TINY
    bad = ok & ~((got - exact).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), g[bad][:4], got[bad][:4], exact[bad][:4])
    return h, r, closed


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate,parts", [("full", False), ("full", True), ("row", False), ("row", True)])
@pytest.mark.parametrize("T,D", [(7, 301), (50, 9), (3, 8300)])
def test_gates_up_to_15(T, D, gate, parts, dtype):
    check(T, D, dtype, gate, parts, T + D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["row", "full"])
def test_gates_to_80(gate, dtype):
    """Without norms and scale dgate = dy f s (1 - s), its factors known in closed form."""
    h = make(90, 40, dtype, gate=gate, post=False, alpha=False, pre=False, seed=3)
    h["gate"] = torch.linspace(-80.0, 80.0, h["gate"].numel()).view_as(h["gate"]).to(dtype)
    d = dev(h)
    r = bwd(d, fwd(d))
    g = h["gate"].double()
    t = h["dy"].double() * h["f"].double()
    m = t.abs()
    if gate == "row":
        t, m = t.sum(1, keepdim=True), m.sum(1, keepdim=True)
    k = torch.sigmoid(g) * torch.sigmoid(-g)
    got = r["dgate"].cpu().double()
    # the sigmoid's (|gate| + 3) twice, a product or two, and for a gate per token the row sum
    tol = (2 * (g.abs() + 3) + 4 + ROW) * ref64.U * m * k + ref64.HALF_STEP[dtype] * (t * k).abs() + ref64.TINY
    bad = ~((got - t * k).abs() <= tol)
    assert not bool(bad.any()), (int(bad.sum()), h["gate"][bad][:4], got[bad][:4], (t * k)[bad][:4])
