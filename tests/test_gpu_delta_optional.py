"""det_delta_rule and its backward with each optional tensor left out, in both forms of the chains, and over
sequences of many chunks."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64_delta as R
from tests.test_gpu_delta_rule import BF, F32, X, bwd, compare, fwd, make, to_dev

pytestmark = pytest.mark.gpu

MANY = [0, 0, 1, 65, 66, 130, 197, 240, 241, 300, 330, 331, 333, 395, 400, 470]   # 15 sequences
FEW = [0, 33, 33, 200]


def only(d, **kw):
    """The forward with nothing but what is named."""
    o = torch.full_like(d["v"], 7.0)
    dg.det_delta_rule(*(d[n] for n in X), o, d["offs"], **kw)
    return o


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 64), (100, 90), (64, 40), (128, 17)])
@pytest.mark.parametrize("offs,H", [(FEW, 2), (MANY, 6)])
def test_outputs_do_not_depend_on_what_else_is_asked_for(offs, H, dk, dv, dtype):
    """(MANY x 6 heads take eight waves for a head's columns, FEW x 2 teams.)"""
    T = offs[-1] + 3
    h = make(T, offs, H // 2, H, dk, dv, dtype, seed=dk + dv)
    d = to_dev(h)
    f = fwd(d)
    s1 = torch.full_like(f["s1"], 7.0)
    assert torch.equal(only(d, initial_state=d["s0"], final_state=s1), f["o"]) and torch.equal(s1, f["s1"])
    assert torch.equal(only(d, initial_state=d["s0"]), f["o"])
    states = torch.full_like(f["states"], 7.0)
    assert torch.equal(only(d, initial_state=d["s0"], states=states), f["o"])
    some = ~torch.isnan(f["states"])    # the rest is left as it was
    assert torch.equal(states[some], f["states"][some]) and (states[~some] == 7.0).all()
    # no initial state is one of zeros
    z = dict(d, s0=torch.zeros_like(d["s0"]), ds1=torch.zeros_like(d["ds1"]))
    fz = fwd(z)
    assert torch.equal(only(d, final_state=s1), fz["o"]) and torch.equal(s1, fz["s1"])
    assert torch.equal(only(d), fz["o"])
    # and no gradient of the final state one of zeros; the initial state's is left out
    r = bwd(z, fz)
    g = {n: torch.full_like(x, 7.0) for n, x in r.items() if n != "ds0"}
    for ds0 in (None, torch.full_like(r["ds0"], 7.0)):
        dg.det_delta_rule_bwd(d["do"], *(d[n] for n in X), d["offs"], fz["states"], g["dq"], g["dk"], g["dv"], g["dg"],
                              g["dbeta"], dinitial_state=ds0)
        for n in g:
            assert torch.equal(g[n], r[n]), n
        assert ds0 is None or torch.equal(ds0, r["ds0"])
    # against 64 bits, in the form that has no states
    o, s1w, mags, _ = R.delta(*(h[n] for n in X), offs, h["s0"], dk ** -0.5)
    n = R.allowed(max(y - x for x, y in zip(offs, offs[1:])) / 32)
    compare(only(d, initial_state=d["s0"], final_state=s1), o, mags["o"], n, "o", 7.0)
    compare(s1, s1w, mags["s1"], n, "final_state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H,offs", [(2, [0, 1, 3000, 3001]), (28, [0, 0, 700, 1500])])
def test_many_chunks(H, offs, dtype):
    """A state that is kept over thousands of tokens and dozens of chunks, and its gradient. Errors are independent from
    chunk to chunk: in the norm of all outputs they are at most two of the standard deviations that one by one eight are
    allowed of (see ref64_delta)."""
    T, dk, dv = offs[-1], 32, 32
    h = make(T, offs, 1, H, dk, dv, dtype, seed=T, g_scale=0.01)
    d = to_dev(h)
    o, s1, mags, kept = R.delta(*(h[n] for n in X), offs, h["s0"], dk ** -0.5)
    n = R.allowed(T / 32)
    f = fwd(d)
    want, more = R.delta_bwd(h["do"], kept, h["ds1"], H)
    got = dict(bwd(d, f), o=f["o"], s1=f["s1"])
    want.update(o=o, s1=s1)
    mags.update(more)
    for name in want:
        m = n if name in ("o", "s1") else 2 * n
        compare(got[name], want[name], mags[name], m, name)
        off = (got[name].cpu().double() - want[name]).norm()
        half = torch.finfo(got[name].dtype).eps / 2
        assert off <= m / 4 * 2.0 ** -24 * mags[name].norm() + half * want[name].norm(), name
