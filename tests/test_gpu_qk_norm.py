"""det_qk_norm and its backward against float64: head sizes from one channel on, every
norm, both pairings, partial rotations, several axes, far positions, strides; parameter
gradients; run-to-run bits; graphs; streams."""
import math

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64_delta as R
from tests.gpu_util import SideLoad
from tests.test_gpu_delta_rule import spaced

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# Roundings on a row's path: its sum of squares 16 + 6 (halved by the root) and the factor 5; the weight and the
# factor 2; cos and sin 4 (their argument, kept in whole turns, 3) and the turn's two products 3. Backward: twice.
FWD, BWD = 30, 90


def make(T, Hq, Hk, D, dtype, R_=0, axes=1, w=True, seed=0, scale=1.0, far=1 << 20):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    h = dict(q=(scale * n(T, Hq, D)).to(dtype), k=(scale * n(T, Hk, D)).to(dtype), dyq=n(T, Hq, D).to(dtype),
             dyk=n(T, Hk, D).to(dtype), w_q=1 + 0.2 * n(D) if w else None, w_k=1 + 0.2 * n(D) if w else None,
             pos=None, inv_freq=None, axis=None)
    if R_:
        h["inv_freq"] = (10000.0 ** (-torch.arange(0, R_, 2, dtype=torch.float64) / R_)).float()
        h["pos"] = torch.randint(-far, far, (axes, T) if axes > 1 else (T,), generator=gen, dtype=torch.int32)
        if axes > 1:
            h["axis"] = torch.randint(0, axes, (R_ // 2,), generator=gen, dtype=torch.int32)
    return h


def to_dev(h, extra=0):
    return {n: None if x is None else spaced(x, extra) if x.dim() == 3 else x.cuda() for n, x in h.items()}


def run(d, norm, eps, pairs, start=0.0, ws=None, stream=None, out=None):
    kw = dict(norm=norm, eps=eps, pos=d["pos"], inv_freq=d["inv_freq"], axis=d["axis"], pairs=pairs, stream=stream)
    o = out or dict({"y" + n: torch.full_like(d[n], 7.0) for n in "qk"}, **{"d" + n: torch.full_like(d[n], 7.0) for n in "qk"},
                    **{"dw_" + n: None if d["w_" + n] is None else torch.full_like(d["w_" + n], start) for n in "qk"})
    dg.det_qk_norm(d["q"], d["k"], o["yq"], o["yk"], w_q=d["w_q"], w_k=d["w_k"], **kw)
    dg.det_qk_norm_bwd(d["dyq"], d["dyk"], d["q"], d["k"], o["dq"], o["dk"], w_q=d["w_q"], w_k=d["w_k"], dw_q=o["dw_q"],
                       dw_k=o["dw_k"], ws=ws, **kw)
    return o


def check(T, Hq, Hk, D, dtype, R_=0, norm="rms", eps=1e-6, pairs="halves", extra=0, start=0.0, **kw):
    h = make(T, Hq, Hk, D, dtype, R_, **kw)
    d = to_dev(h, extra)
    o = run(d, norm, eps, pairs, start)
    cs = R.turns(h["pos"], h["inv_freq"], h["axis"]) if R_ else None
    for n in "qk":
        y, mag = R.qk(h[n], h["w_" + n], norm, eps, cs, pairs)
        R.assert_close(o["y" + n], y, mag, FWD, "y" + n)
        dx, mag, dw, dw_mag = R.qk_bwd(h["dy" + n], h[n], h["w_" + n], norm, eps, cs, pairs)
        R.assert_close(o["d" + n], dx, mag, BWD, "d" + n)
        if h["w_" + n] is not None:
            rows = T * h[n].shape[1]     # a lane's chain at the most, then its wave and workgroup
            R.assert_close(o["dw_" + n], dw + start, dw_mag + abs(start), BWD + min(rows, 600) + 12, "dw_" + n)
    return d, o


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("D,R_", [(1, 0), (2, 2), (3, 2), (7, 4), (8, 8), (15, 6), (16, 16), (17, 16), (32, 16), (34, 34),
                                  (64, 64), (80, 40), (96, 96), (100, 30), (127, 126), (128, 128), (128, 64), (128, 32),
                                  (192, 64), (250, 250), (256, 256), (512, 512), (513, 512), (1000, 500), (1024, 1024)])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_head_sizes(D, R_, pairs, dtype):
    check(21, 3, 2, D, dtype, R_, pairs=pairs, seed=D)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("w", [False, True])
@pytest.mark.parametrize("R_", [0, 40])
def test_norms(norm, w, R_, dtype):
    check(50, 4, 1, 72, dtype, R_, norm=norm, w=w, start=1.5 if w else 0.0)


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 64, 8), (3, 1, 5), (1023, 2, 1), (1025, 7, 3), (5000, 5, 1)])
def test_tokens_and_heads(T, Hq, Hk):
    check(T, Hq, Hk, 64, BF, 64)
    check(T, Hq, Hk, 48, F32, 20, norm="l2")


@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
@pytest.mark.parametrize("axes", [2, 3, 5])
def test_axes(axes, pairs):
    check(40, 3, 2, 128, F32, 128, axes=axes, pairs=pairs, seed=axes)


def test_far_positions():
    """All of int32: the angle keeps its digits."""
    check(64, 1, 1, 64, F32, 64, far=(1 << 31) - 1, norm="none", w=False)


def test_an_axis_that_there_is_not_turns_nothing():
    h = make(10, 1, 1, 16, F32, 16, axes=2, w=False)
    h["axis"] = torch.tensor([0, 1, 2, -1, 7, 0, 1, 1 << 30], dtype=torch.int32)
    d = to_dev(h)
    o = run(d, "none", 0.0, "neighbours")
    for p in (2, 3, 4, 7):
        assert torch.equal(o["yq"][..., 2 * p:2 * p + 2], d["q"][..., 2 * p:2 * p + 2])
    y, mag = R.qk(h["q"], None, "none", 0.0, R.turns(h["pos"], h["inv_freq"], h["axis"]), "neighbours")
    R.assert_close(o["yq"], y, mag, FWD, "y")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(dtype):
    check(33, 3, 2, 128, dtype, 128, extra=5)
    check(33, 3, 2, 50, dtype, 20, extra=3)


def test_column_ranges_of_one_buffer():
    """q and k as ranges of one projection's output, the outputs ranges of another buffer, as the gradients are."""
    h = make(30, 4, 2, 64, BF, 64)
    qkv = torch.zeros(30, 8, 64, dtype=BF, device="cuda")
    qkv[:, :4], qkv[:, 4:6] = h["q"].cuda(), h["k"].cuda()
    d = dict(to_dev(h), q=qkv[:, :4], k=qkv[:, 4:6])
    out, grad = torch.zeros_like(qkv), torch.full_like(qkv, 3.0)
    o = run(to_dev(h), "rms", 1e-6, "halves")
    e = run(d, "rms", 1e-6, "halves", out=dict(yq=out[:, :4], yk=out[:, 4:6], dq=grad[:, :4], dk=grad[:, 4:6],
                                               dw_q=torch.zeros(64, device="cuda"), dw_k=torch.zeros(64, device="cuda")))
    for n in o:
        assert torch.equal(o[n], e[n]), n
    assert (out[:, 6:] == 0).all() and (grad[:, 6:] == 3.0).all()


def test_one_side_alone():
    h = make(20, 3, 2, 64, F32, 32)
    d = to_dev(h)
    o = run(d, "rms", 1e-6, "halves")
    kw = dict(pos=d["pos"], inv_freq=d["inv_freq"])
    for n, other in (("q", "k"), ("k", "q")):
        y, g, dw = torch.zeros_like(d[n]), torch.zeros_like(d[n]), torch.zeros(64, device="cuda")
        a = (d[n], None, y, None) if n == "q" else (None, d[n], None, y)
        dg.det_qk_norm(*a, **{"w_" + n: d["w_" + n]}, **kw)
        a = (d["dy" + n], None, d[n], None, g, None) if n == "q" else (None, d["dy" + n], None, d[n], None, g)
        dg.det_qk_norm_bwd(*a, **{"w_" + n: d["w_" + n], "dw_" + n: dw}, **kw)
        assert torch.equal(y, o["y" + n]) and torch.equal(g, o["d" + n])
        R.assert_close(dw, o["dw_" + n].cpu().double(), o["dw_" + n].cpu().double().abs() + 60, 100, "dw")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_zeros_and_extremes(dtype):
    h = make(6, 1, 1, 32, dtype, 0)
    h["q"][0] = 0.0
    h["q"][1] = 1e-20
    h["q"][2, 0, 3] = math.nan
    h["q"][3, 0, 3] = math.inf
    d = to_dev(h)
    o = run(d, "rms", 1e-6, "halves")
    assert (o["yq"][0] == 0).all()
    y, mag = R.qk(h["q"], h["w_q"], "rms", 1e-6, None, "halves")
    R.assert_close(o["yq"][1], y[1], mag[1], FWD, "tiny")
    assert torch.isnan(o["yq"][2]).all() and torch.isnan(o["yq"][3, 0, 3])
    R.assert_close(o["yq"][4:], y[4:], mag[4:], FWD, "others")


@pytest.mark.parametrize("norm", ["rms", "l2", "none"])
@pytest.mark.parametrize("pairs", ["halves", "neighbours"])
def test_gradients_against_differences(norm, pairs):
    """Central differences of the float64 formula, whose gradient the kernels' is held to elsewhere: off by the third
    derivative's eps^2, here below 1e-8 of the sum of the terms' sizes."""
    h = make(6, 2, 1, 24, F32, 16, axes=2, seed=3)
    cs = R.turns(h["pos"], h["inv_freq"], h["axis"])
    o = run(to_dev(h), norm, 1e-6, pairs)
    gen = torch.Generator().manual_seed(1)
    for n in "qk":
        x, w, dy = h[n].double(), h["w_" + n].double(), h["dy" + n].double()
        f = lambda x, w: (R.qk(x, w, norm, 1e-6, cs, pairs)[0] * dy).sum()  # noqa: E731
        u, m = torch.randn(x.shape, generator=gen).double(), torch.randn(w.shape, generator=gen).double()
        _, dx_mag, _, dw_mag = R.qk_bwd(h["dy" + n], h[n], h["w_" + n], norm, 1e-6, cs, pairs)
        e = 1e-5
        for got, diff, mag in (((o["d" + n].cpu().double() * u).sum(), (f(x + e * u, w) - f(x - e * u, w)) / (2 * e), (dx_mag * u.abs()).sum()),
                               ((o["dw_" + n].cpu().double() * m).sum(), (f(x, w + e * m) - f(x, w - e * m)) / (2 * e), (dw_mag * m.abs()).sum())):
            assert abs(got - diff) <= (BWD + 20) * 2.0 ** -24 * mag + 1e-8 * mag, n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replay_under_load_with_poisoned_workspaces(dtype):
    d = to_dev(make(3001, 8, 2, 128, dtype, 128))
    load, first = SideLoad(64, 4), None
    need = dg.det_qk_norm_bwd_workspace_size(3001, 8, 2, 128)
    for i in range(8):
        load.kick()
        ws = torch.full((need // 4,), (math.nan, 3e38, -1.0)[i % 3], device="cuda").view(torch.uint8)
        o = run(d, "rms", 1e-6, "halves", start=0.5, ws=ws)
        first = first or {n: x.clone() for n, x in o.items()}
        assert all(torch.equal(first[n], o[n]) for n in o)
    load.wait()


def test_graph_replays_and_two_streams():
    d = to_dev(make(2000, 8, 2, 128, BF, 128, axes=3))
    want = {n: x.clone() for n, x in run(d, "rms", 1e-6, "halves").items()}
    g, o = torch.cuda.CUDAGraph(), run(d, "rms", 1e-6, "halves")
    with torch.cuda.graph(g):
        run(d, "rms", 1e-6, "halves", out=o)
    for i in range(4):
        for n, x in o.items():
            x.fill_(0.0 if n.startswith("dw") else float(i))
        g.replay()
        e = run(d, "rms", 1e-6, "halves")
        torch.cuda.synchronize()
        assert all(torch.equal(o[n], want[n]) and torch.equal(e[n], want[n]) for n in o)
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        o = {n: torch.zeros_like(x) for n, x in want.items()}
        torch.cuda.synchronize()
        run(d, "rms", 1e-6, "halves", out=o, stream=s)
        outs.append(o)
    torch.cuda.synchronize()
    assert all(torch.equal(o[n], want[n]) for o in outs for n in o)


def test_large_outputs_past_the_caches():
    """Outputs of 256 MiB and more are stored another way: the same bits as in two halves."""
    T = 33000
    q = torch.randn(T, 32, 128, device="cuda", dtype=BF)
    pos, f = torch.arange(T, device="cuda", dtype=torch.int32), (10000.0 ** (-torch.arange(0, 64, device="cuda") / 64.0))
    y, y2 = torch.zeros_like(q), torch.zeros_like(q)
    dg.det_qk_norm(q, None, y, None, pos=pos, inv_freq=f)
    for a in (slice(0, T // 2), slice(T // 2, T)):
        dg.det_qk_norm(q[a], None, y2[a], None, pos=pos[a], inv_freq=f)
    assert torch.equal(y, y2)
    dx, dx2 = torch.zeros_like(q), torch.zeros_like(q)
    dg.det_qk_norm_bwd(y, None, q, None, dx, None, pos=pos, inv_freq=f)
    for a in (slice(0, T // 2), slice(T // 2, T)):
        dg.det_qk_norm_bwd(y2[a], None, q[a], None, dx2[a], None, pos=pos[a], inv_freq=f)
    assert torch.equal(dx, dx2)
