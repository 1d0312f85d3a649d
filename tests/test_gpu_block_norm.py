"""det_block_norm and its backward against float64, with every combination of
optional parts, odd widths, strides and scales; run-to-run bits; graphs; streams."""
import itertools
import math

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64
from tests.gpu_util import SideLoad, note
from tests.test_gpu_router_balance import strided

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NAMES = ("x", "f", "gate", "w_post", "alpha", "w_pre", "dy", "dh")


def make(T, D, dtype, gate="full", post=True, alpha=True, pre=True, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)

    def rows(cols, s=1.0):
        return (torch.randn(T, cols, generator=g) * s).to(dtype)

    def vec():
        return torch.randn(D, generator=g)
    return dict(x=rows(D, scale), f=rows(D, scale), gate=None if gate == "none" else rows(D if gate == "full" else 1, 2.0),
                w_post=vec() if post else None, alpha=vec() if alpha else None, w_pre=vec() if pre else None,
                dy=rows(D), dh=rows(D) if pre else None)


def dev(d, ld_extra=0, shift=0):
    out = {}
    for k, v in d.items():
        if v is None:
            out[k] = None
        elif v.dim() == 2 and (ld_extra or shift):
            out[k] = strided(v, v.shape[1] + ld_extra, shift)
        else:
            out[k] = v.cuda()
    return out


def like(t, fill=9.0):
    return None if t is None else torch.full_like(t, fill)


def fwd(d, eps=1e-6, stream=None, outs=None):
    T = d["x"].shape[0]
    o = outs or dict(y=like(d["x"]), h=like(d["x"]) if d["w_pre"] is not None else None,
                     rstd_post=torch.full((T,), 9.0, device="cuda") if d["w_post"] is not None else None,
                     rstd_pre=torch.full((T,), 9.0, device="cuda") if d["w_pre"] is not None else None)
    dg.det_block_norm(d["x"], d["f"], o["y"], gate=d["gate"], w_post=d["w_post"], alpha=d["alpha"], w_pre=d["w_pre"],
                      h=o["h"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"], eps=eps, stream=stream)
    return o


def bwd(d, o, start=0.0, ws=None, stream=None):
    D = d["f"].shape[1]
    r = dict(dx=like(d["dy"]), df=like(d["dy"]), dgate=like(d["gate"]))
    for n in ("w_post", "alpha", "w_pre"):
        r["d" + n] = None if d[n] is None else torch.full((D,), start, device="cuda")
    dg.det_block_norm_bwd(d["dy"], d["x"], d["f"], r["dx"], r["df"], dh=d["dh"], gate=d["gate"], w_post=d["w_post"],
                          alpha=d["alpha"], w_pre=d["w_pre"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"],
                          dgate=r["dgate"], dw_post=r["dw_post"], dalpha=r["dalpha"], dw_pre=r["dw_pre"], ws=ws,
                          stream=stream)
    return r


# Roundings on a row's path. A row sum: a lane's chain of at most 16, its tree of 6, 16 waves: 38; a norm's factor
# 38 / 2 + 4; the sigmoid's exponent and quotient 6; products and sums 8 each way. A column sum: at most 64 rows of a
# workgroup here, 16 + 6 slots.
ROW, COL = 38, 64 + 22


def check(T, D, dtype, ld_extra=0, shift=0, eps=1e-6, start=0.0, **kw):
    h = make(T, D, dtype, **kw)
    d = dev(h, ld_extra, shift)
    o = fwd(d, eps)
    w = ref64.norm(h["x"], h["f"], h["gate"], h["w_post"], h["alpha"], h["w_pre"], eps)
    n = ROW + 30
    ref64.assert_close(o["y"], w["y"], w["y_mag"], n, "y")
    if h["w_post"] is not None:
        ref64.assert_close(o["rstd_post"], w["rstd_post"], w["rstd_post"], n, "rstd_post")
    if h["w_pre"] is not None:
        big = (1 + w["pre_mag"])
        ref64.assert_close(o["rstd_pre"], w["rstd_pre"], w["rstd_pre"] * big, n, "rstd_pre")
        ref64.assert_close(o["h"], w["h"], w["h_mag"] + w["h"].abs() * big[:, None], n, "h")
    r = bwd(d, o, start)
    rs = {k: None if o[k] is None else o[k].cpu() for k in ("rstd_post", "rstd_pre")}
    w = ref64.norm_bwd(h["dy"], h["dh"], h["x"], h["f"], h["gate"], h["w_post"], h["alpha"], h["w_pre"],
                       rs["rstd_post"], rs["rstd_pre"])
    n = 2 * ROW + 60
    for k, v in r.items():
        if v is None:
            continue
        if k in ("dx", "df", "dgate"):
            # a gate per token: its D terms carry the row's roundings and add a chain of their own
            ref64.assert_close(v, w[k], w[k + "_mag"], n + (ROW if k == "dgate" else 0), k)
        else:
            ref64.assert_close(v, w[k] + start, w[k + "_mag"] + abs(start), n + COL, k)
    return d, o, r


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(1, 1), (3, 1), (2, 2), (5, 7), (4, 8), (3, 9), (130, 64), (9, 511), (6, 512),
                                 (7, 513), (5, 1000), (4, 1024), (3, 1407), (5, 2048), (2, 2056), (3, 4096),
                                 (2, 5000), (3, 8192), (2, 8193), (3, 16384)])
def test_sizes(T, D, dtype):
    check(T, D, dtype, seed=T + D)


@pytest.mark.parametrize("gate", ["none", "row", "full"])
@pytest.mark.parametrize("post,alpha,pre", list(itertools.product([False, True], repeat=3)))
def test_every_combination_of_parts(gate, post, alpha, pre):
    check(37, 203, F32, gate=gate, post=post, alpha=alpha, pre=pre, seed=1, start=2.5)
    check(5, 1030, BF, gate=gate, post=post, alpha=alpha, pre=pre, seed=2)


@pytest.mark.parametrize("gate,post,alpha,pre", [("none", True, False, True), ("row", False, True, True),
                                                 ("full", True, True, False), ("row", True, True, True),
                                                 ("none", False, False, False), ("full", False, False, True)])
def test_wide_rows(gate, post, alpha, pre):
    """More than 8192 channels: sixteen per thread, one workgroup walking several rows."""
    check(5, 8200, F32, gate=gate, post=post, alpha=alpha, pre=pre, seed=3)
    check(600, 9001, BF, gate=gate, post=post, alpha=alpha, pre=pre, seed=4, ld_extra=3, shift=1)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gate", ["row", "full"])
def test_strides_and_unaligned_rows(gate, dtype):
    d, o, r = check(21, 331, dtype, ld_extra=6, shift=3, gate=gate, seed=3)
    # outputs with strides of their own: the same bits, and nothing written beside the rows
    y, h = (strided(torch.zeros(21, 331, dtype=dtype), 340, 1) for _ in range(2))
    o2 = fwd(d, outs=dict(o, y=y, h=h))
    assert torch.equal(o2["y"], o["y"]) and torch.equal(o2["h"], o["h"])
    for t in (y, h):
        assert bool((t._base[1:].view(-1)[:21 * 340].view(21, 340)[:, 331:] == 77).all())


@pytest.mark.parametrize("scale", [1e-12, 1e-3, 1e6, 1e15])
def test_scales(scale):
    """Rows far below eps and far above one (their squares stay inside float32)."""
    check(9, 300, F32, seed=4, scale=scale, eps=1e-6)


def test_zero_rows_and_extreme_gates():
    h = make(6, 70, F32, seed=5)
    h["f"][0] = 0
    h["x"][1] = 0
    h["f"][1] = 0
    h["gate"][2] = math.inf
    h["gate"][3] = -math.inf
    h["gate"][4] = torch.finfo(F32).min
    h["gate"][5] = 100.0
    d = dev(h)
    o = fwd(d)
    w = ref64.norm(h["x"], h["f"], h["gate"], h["w_post"], h["alpha"], h["w_pre"], 1e-6)
    ref64.assert_close(o["y"], w["y"], w["y_mag"], 80, "y")
    assert torch.equal(o["y"][3], d["x"][3]) and bool((o["h"][1] == 0).all())
    r = bwd(d, o)
    assert all(bool(torch.isfinite(v).all()) for v in r.values())
    assert bool((r["dgate"][2:5] == 0).all()) and bool((r["df"][3:5] == 0).all())


def test_nan_stays_in_its_row():
    h = make(50, 130, F32, seed=6)
    d = dev(h)
    clean = fwd(d)
    d["f"][7, 3] = math.nan
    o = fwd(d)
    bad = torch.isnan(o["y"]).any(1).nonzero().flatten().tolist()
    assert bad == [7] and torch.equal(o["h"][:7], clean["h"][:7]) and torch.equal(o["h"][8:], clean["h"][8:])
    r = bwd(d, o)
    assert torch.isnan(r["dx"]).any(1).nonzero().flatten().tolist() == [7]


def test_no_tokens():
    h = make(0, 16, F32)
    d = dev(h)
    r = bwd(d, fwd(d), start=3.0)
    assert all(bool((r[k] == 3).all()) for k in ("dw_post", "dalpha", "dw_pre"))


def test_gradients_against_differences():
    """Every input's gradient of sum(y cy + h ch), against central differences of the float64 forward."""
    for gate in ("row", "full"):
        h = make(3, 6, F32, gate=gate, seed=7)
        d = dev(h)
        r = bwd(d, fwd(d))
        step = 1e-5

        def total(c):
            w = ref64.norm(c["x"], c["f"], c["gate"], c["w_post"], c["alpha"], c["w_pre"], 1e-6)
            return float((w["y"] * h["dy"].double()).sum() + (w["h"] * h["dh"].double()).sum())
        for k in ("x", "f", "gate", "w_post", "alpha", "w_pre"):
            for i in range(h[k].numel()):
                v = []
                for s in (step, -step):
                    c = dict(h)
                    c[k] = h[k].double().clone()
                    c[k].view(-1)[i] += s
                    v.append(total(c))
                got = float(r["d" + k].flatten()[i])
                assert abs((v[0] - v[1]) / (2 * step) - got) < 1e-4 * (1 + abs(got)), (gate, k, i)


def test_parameter_gradients_accumulate_over_microbatches():
    h = make(64, 96, F32, seed=8)
    d = dev(h)
    o = fwd(d)
    once, twice = bwd(d, o), bwd(d, o, start=1.0)
    for k in ("dw_post", "dalpha", "dw_pre"):
        assert torch.equal(twice[k], once[k] + 1.0)    # RN32(out + total), the same total


def test_long_columns():
    """More tokens than one slot holds: 20011 rows, against float64. A workgroup adds at most 20011 / 256 rows."""
    h = make(20011, 72, BF, seed=9)
    d = dev(h)
    o = fwd(d)
    r = bwd(d, o)
    rs = {k: o[k].cpu() for k in ("rstd_post", "rstd_pre")}
    w = ref64.norm_bwd(h["dy"], h["dh"], h["x"], h["f"], h["gate"], h["w_post"], h["alpha"], h["w_pre"],
                       rs["rstd_post"], rs["rstd_pre"])
    for k in ("dw_post", "dalpha", "dw_pre"):
        ref64.assert_close(r[k], w[k], w[k + "_mag"], 2 * ROW + 60 + 80 + 300, k)


def test_rows_past_32_bit_offsets():
    ld, D = (1 << 30) + 8, 260

    def far(t):
        v = torch.empty(2 * ld + D, dtype=BF, device="cuda").as_strided((3, t.shape[1]), (ld, 1))
        v.copy_(t)
        return v
    h = make(3, D, BF, seed=10)
    near = dev(h)
    d = {k: far(v) if v is not None and v.dim() == 2 else near[k] for k, v in h.items()}
    want = fwd(near)
    outs = dict(y=far(torch.zeros(3, D)), h=far(torch.zeros(3, D)), rstd_post=torch.zeros(3, device="cuda"),
                rstd_pre=torch.zeros(3, device="cuda"))
    o = fwd(d, outs=outs)
    assert all(torch.equal(o[k], want[k]) for k in want)
    a = bwd(near, want)
    r = dict(dx=far(torch.zeros(3, D)), df=far(torch.zeros(3, D)), dgate=far(torch.zeros(3, D)))
    g = [torch.zeros(D, device="cuda") for _ in range(3)]
    dg.det_block_norm_bwd(d["dy"], d["x"], d["f"], r["dx"], r["df"], dh=d["dh"], gate=d["gate"], w_post=d["w_post"],
                          alpha=d["alpha"], w_pre=d["w_pre"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"],
                          dgate=r["dgate"], dw_post=g[0], dalpha=g[1], dw_pre=g[2])
    assert all(torch.equal(r[k], a[k]) for k in r)
    assert torch.equal(g[0], a["dw_post"]) and torch.equal(g[1], a["dalpha"]) and torch.equal(g[2], a["dw_pre"])


@pytest.mark.parametrize("dtype,T,D", [(BF, 8200, 8192), (F32, 12001, 3001)])
def test_outputs_past_the_caches(dtype, T, D):
    """Outputs larger than the last-level cache are stored another way: every row has the bits of a small call, and the
    parameter gradients agree with float64 column sums of the call's own rows."""
    assert 2 * T * D * torch.finfo(dtype).bits // 8 >= 256 << 20
    g = torch.Generator(device="cuda").manual_seed(2)

    def rows(n):
        return torch.randn(n, D, device="cuda", dtype=dtype, generator=g)
    d = dict(x=rows(T), f=rows(T), gate=rows(T), dy=rows(T), dh=rows(T),
             **{k: 1 + 0.1 * torch.randn(D, device="cuda", generator=g) for k in ("w_post", "alpha", "w_pre")})
    o = fwd(d)
    r = bwd(d, o)
    for a in range(0, T, 1499):
        e = {k: v[a:a + 5] if v.dim() == 2 else v for k, v in d.items()}
        p = fwd(e)
        assert all(torch.equal(p[k], o[k][a:a + 5]) for k in o), a
        q = bwd(e, p)
        assert all(torch.equal(q[k], r[k][a:a + 5]) for k in ("dx", "df", "dgate")), a
    # dw_pre = sum dh yh from the stored y (off by half a step each) and the call's factors
    yh = o["y"].double() * o["rstd_pre"].double()[:, None]
    want, mag = (d["dh"].double() * yh).sum(0), (d["dh"].double() * yh).abs().sum(0)
    tol = (ref64.HALF_STEP[dtype] + 400 * ref64.U) * mag
    assert bool(((r["dw_pre"].double() - want).abs() <= tol).all())


def test_backward_without_x():
    """x enters the backward only through the second norm."""
    h = make(40, 150, F32, pre=False, seed=20)
    d = dev(h)
    o = fwd(d)
    want = bwd(d, o)
    got = bwd(dict(d, x=None), o)
    assert all(v is None or torch.equal(v, got[k]) for k, v in want.items())


def test_replay_under_load_with_poisoned_workspaces():
    d = dev(make(3000, 640, BF, gate="row", seed=11))
    n = dg.det_block_norm_bwd_workspace_size(3000, 640)
    first, load = None, SideLoad(mib=64, iters=4)
    for fill in (0, 255, 127, 1, 255, 3, 0, 90):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        ws = ws[-ws.data_ptr() % 256:][:n]
        load.kick()
        o = fwd(d)
        got = [v.clone() for v in (*o.values(), *bwd(d, o, ws=ws).values()) if v is not None]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        assert bool((ws[:256] == fill).all())
    load.wait()
    note("block norm: 8 runs under load with poisoned workspaces, same bits")


def test_graph_replays_and_two_streams():
    d = dev(make(700, 384, BF, seed=12))
    o = fwd(d)
    dx, df, dgate = (torch.zeros_like(d["dy"]) for _ in range(3))
    dw = torch.zeros(3, 384, device="cuda")

    def step():
        fwd(d, outs=o)
        dg.det_block_norm_bwd(d["dy"], d["x"], d["f"], dx, df, dh=d["dh"], gate=d["gate"], w_post=d["w_post"],
                              alpha=d["alpha"], w_pre=d["w_pre"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"],
                              dgate=dgate, dw_post=dw[0], dalpha=dw[1], dw_pre=dw[2])
    outs = [o["y"], o["h"], o["rstd_post"], o["rstd_pre"], dx, df, dgate, dw]
    graphs = []
    for _ in range(2):
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for r in range(4):
        d["f"].mul_(0.9)
        dw.fill_(0.5)
        step()
        want = [t.clone() for t in outs]
        for g in graphs:
            for t in outs:
                t.fill_(7)
            dw.fill_(0.5)
            torch.empty(1 << 20, device="cuda").normal_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), r
    # two streams at once, each call with a workspace of its own
    want = bwd(d, o)
    torch.cuda.synchronize()
    res = []
    for r in range(4):
        for s in [torch.cuda.Stream() for _ in range(2)]:
            with torch.cuda.stream(s):
                res.append(bwd(d, o, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(v, want[k]) for q in res for k, v in q.items())
