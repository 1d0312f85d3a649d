"""det_delta_rule, its backward and its single-token form against float64: lengths from
zero on, odd head sizes, shared key heads, strides, strong decays, empty sequences;
gradients against differences; run-to-run bits; graphs; streams."""
import math

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64_delta as R
from tests.gpu_util import SideLoad

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, offs, Hk, H, dk, dv, dtype, seed=0, g_scale=1.0, init=True, unit=True):
    gen = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, k = n(T, Hk, dk) + 0.5 * n(1, Hk, dk), n(T, Hk, dk) + 0.5 * n(1, Hk, dk)
    if unit:
        q, k = (x / x.norm(dim=-1, keepdim=True) for x in (q, k))
    S = len(offs) - 1
    return dict(q=q.to(dtype), k=k.to(dtype), v=n(T, H, dv).to(dtype), g=-g_scale * torch.rand(T, H, generator=gen) ** 3,
                beta=torch.sigmoid(1.5 * n(T, H)).to(dtype), offs=torch.tensor(offs, dtype=torch.int32),
                s0=0.3 * n(S, H, dk, dv) if init else None, do=n(T, H, dv).to(dtype), ds1=0.1 * n(S, H, dk, dv) if init else None)


def spaced(x, extra):
    """x on the GPU as a column range of wider tokens, off the start of the allocation by an odd number of elements."""
    if not extra or x.dim() < 2 or x.shape[0] == 0:
        return x.cuda()
    width = x[0].numel()
    buf = torch.full((3 + x.shape[0] * (width + extra),), 55.0, device="cuda").to(x.dtype)
    v = buf[3:].view(x.shape[0], width + extra)[:, :width].unflatten(1, x.shape[1:])
    v.copy_(x)
    return v


def to_dev(h, extra=0):
    return {n: None if x is None else x.cuda() if n in ("offs", "s0", "ds1") else spaced(x, extra) for n, x in h.items()}


X = ("q", "k", "v", "g", "beta")


def fwd(d, scale=None, states=True, ws=None, stream=None, out=None):
    o = out or dict(o=torch.full_like(d["v"], 7.0),
                    s1=torch.full((len(d["offs"]) - 1, d["v"].shape[1], d["q"].shape[2], d["v"].shape[2]), 7.0, device="cuda"),
                    states=torch.full(dg.det_delta_rule_states_shape(d["q"], d["v"], d["offs"]), math.nan, device="cuda")
                    if states else None)
    dg.det_delta_rule(*(d[n] for n in X), o["o"], d["offs"], initial_state=d["s0"], final_state=o["s1"], states=o["states"],
                      scale=scale, ws=ws, stream=stream)
    return o


def bwd(d, f, scale=None, ws=None, stream=None, out=None):
    r = out or dict({"d" + n: torch.full_like(d[n], 7.0) for n in ("q", "k", "v", "beta")},
                    dg=torch.full_like(d["beta"], 7.0), ds0=torch.full_like(f["s1"], 7.0))
    dg.det_delta_rule_bwd(d["do"], *(d[n] for n in X), d["offs"], f["states"], r["dq"], r["dk"], r["dv"], r["dg"], r["dbeta"],
                          dfinal_state=d["ds1"], dinitial_state=r["ds0"], scale=scale, ws=ws, stream=stream)
    return r


def compare(got, want, mag, n, what, left=None):
    """Rows that no sequence holds (NaN in the reference) keep what was there."""
    assert got.shape == want.shape, what
    none = torch.isnan(want)
    if left is not None and none.any():
        assert (got.detach().cpu().double()[none] == left).all(), what + ": rows behind the sequences"
    R.assert_close(torch.where(none.cuda(), torch.zeros_like(got), got), torch.where(none, torch.zeros_like(want), want), mag,
                   n, what)


def check(T, offs, Hk=1, H=1, dk=64, dv=64, dtype=F32, extra=0, scale=None, back=True, **kw):
    h = make(T, offs, Hk, H, dk, dv, dtype, **kw)
    d = to_dev(h, extra)
    sc = dk ** -0.5 if scale is None else scale
    o, s1, mags, kept = R.delta(*(h[n] for n in X), offs, h["s0"], sc)
    b = R.bounds(offs, T)
    n = R.allowed(max([1] + [y - x for x, y in zip(b, b[1:])]) / 32)
    f = fwd(d, scale)
    compare(f["o"], o, mags["o"], n, "o", 7.0)
    compare(f["s1"], s1, mags["s1"], n, "final_state")
    if back:
        want, mags = R.delta_bwd(h["do"], kept, h["ds1"], H // Hk)
        r = bwd(d, f, scale)
        for name in ("dv", "dq", "dk", "dbeta", "dg", "ds0"):
            compare(r[name], want[name], mags[name], 2 * n, name, 7.0)
    return d, f


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(T, dtype):
    check(T, [0, T], dtype=dtype, seed=T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (16, 16), (31, 33), (64, 128), (128, 64), (65, 1), (1, 128), (100, 90),
                                   (128, 128), (127, 113), (80, 17)])
def test_head_sizes(dk, dv, dtype):
    check(90, [0, 90], H=2, Hk=2, dk=dk, dv=dv, dtype=dtype, seed=dk + dv)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk,H", [(1, 2), (2, 6), (3, 3), (1, 8)])
def test_shared_key_heads(Hk, H, dtype):
    check(140, [0, 75, 140], Hk, H, 48, 40, dtype, seed=H)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("offs", [[0], [0, 0], [0, 0, 0, 70, 70, 150], [5, 60, 200], [-3, 20, 10, 130], [0, 64, 128, 192],
                                  [0, 1, 2, 3, 4], [100, 100]])
def test_packed_sequences(offs, dtype):
    check(160, offs, 1, 2, 32, 48, dtype, seed=len(offs))


def test_many_sequences():
    offs = torch.randint(0, 500, (130,), generator=torch.Generator().manual_seed(1)).sort().values.tolist()
    check(500, [0] + offs, 1, 1, 32, 32, F32, seed=3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("Hk,H,dk,dv,extra", [(3, 6, 128, 128, 0), (6, 6, 64, 64, 0), (2, 6, 100, 90, 0), (6, 6, 64, 128, 5), (6, 6, 128, 50, 0)])
def test_many_chains(Hk, H, dk, dv, extra, dtype):
    """More sequences and heads than take the form for few."""
    offs = [0, 0, 1, 65, 66, 130, 197, 240, 241, 300, 330, 331, 333, 395, 400, 470]
    check(475, offs, Hk, H, dk, dv, dtype, extra=extra, seed=dk)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv,extra", [(128, 128, 0), (64, 50, 3)])
def test_both_forms_give_the_same_bits(dk, dv, extra, dtype):
    """Each sequence alone (few chains) gives its rows of a packed call of many."""
    offs = [0, 150, 150, 214, 300, 301, 330, 400, 401, 402, 430]
    h = make(430, offs, 9, 9, dk, dv, dtype, seed=12)
    d = to_dev(h, extra)
    f = fwd(d)
    r = bwd(d, f)
    for s in (0, 1, 3, 4, 6):
        a, b = offs[s:s + 2]
        e = {n: x[a:b] for n, x in d.items() if n in X + ("do",)}
        e.update(offs=torch.tensor([0, b - a], dtype=torch.int32).cuda(), s0=d["s0"][s:s + 1].contiguous(),
                 ds1=d["ds1"][s:s + 1].contiguous())
        g = fwd(e)
        q = bwd(e, g)
        assert torch.equal(g["o"], f["o"][a:b]) and torch.equal(g["s1"][0], f["s1"][s]), s
        for n in ("dq", "dk", "dv", "dg", "dbeta"):
            assert torch.equal(q[n], r[n][a:b]), (s, n)
        assert torch.equal(q["ds0"][0], r["ds0"][s]), s


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [2, 90])
def test_values_at_any_place(H, dtype):
    """Rows of v and do whose starts or strides are not whole 16 bytes, and tokens far apart, give the same bits."""
    h = make(140, [0, 75, 140], H, H, 64, 48, dtype, seed=13)
    d = to_dev(h)
    f = fwd(d)
    r = bwd(d, f)

    def wide(x):
        y = torch.zeros((140, 1 << 18), dtype=x.dtype, device="cuda")[:, 8:8 + x[0].numel()].unflatten(1, x.shape[1:])
        return y.copy_(x)
    for e in (dict(d, v=spaced(h["v"], 3), do=spaced(h["do"], 5)), dict(d, q=wide(d["q"]), k=wide(d["k"]), v=wide(d["v"]), do=wide(d["do"]))):
        g = fwd(e, out=dict(f, o=spaced(torch.full_like(h["v"], 7.0), 1), s1=f["s1"].clone(), states=f["states"].clone()))
        assert torch.equal(g["o"], f["o"]) and torch.equal(g["s1"], f["s1"])
        for n, x in bwd(e, g).items():
            assert torch.equal(x, r[n]), n


@pytest.mark.parametrize("dtype", [BF, F32])
def test_offsets_past_32_bits(dtype):
    """Tokens 2^24 elements and more apart: the last ones lie past 2^32 bytes."""
    T, H = 140 if dtype == BF else 70, 2
    h = make(T, [0, T], 1, H, 64, 64, dtype, seed=14)
    d = to_dev(h)
    f = fwd(d)
    r = bwd(d, f)

    def far(x, extra=8):
        return torch.empty((T, (1 << 24) + extra), dtype=x.dtype, device="cuda")[:, :x[0].numel()].unflatten(1, x.shape[1:])
    e = dict(d, **{n: far(d[n]).copy_(d[n]) for n in ("q", "k", "v", "do")})
    g = fwd(e, out=dict(f, o=far(d["v"]), s1=f["s1"].clone(), states=f["states"].clone()))
    assert torch.equal(g["o"], f["o"]) and torch.equal(g["s1"], f["s1"])
    for n, x in bwd(e, g, out=dict(r, dq=far(d["q"]), dk=far(d["k"]), dv=far(d["v"]))).items():
        assert torch.equal(x, r[n]), n


def test_no_tokens():
    d, f = check(0, [0, 0, 0], 1, 2, 16, 16, F32)
    assert torch.equal(f["s1"], d["s0"])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_without_states_and_gradients_of_them(dtype):
    check(100, [0, 60, 100], 1, 2, 64, 64, dtype, init=False, scale=0.7)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strides(dtype):
    check(100, [0, 60, 97], 2, 4, 64, 72, dtype, extra=5)


def test_heads_outside_tokens():
    """[H, T, dim] tensors seen as [T, H, dim]."""
    h = make(70, [0, 70], 2, 2, 32, 32, F32)
    d = to_dev(h)
    e = dict(d, **{n: d[n].transpose(0, 1).contiguous().transpose(0, 1) for n in ("q", "k", "v", "do")})
    f0, f1 = fwd(d), fwd(e)
    assert torch.equal(f0["o"], f1["o"])
    for a, b in zip(bwd(d, f0).values(), bwd(e, f1).values()):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("g_scale", [0.0, 20.0, 500.0])
def test_decays(g_scale, dtype):
    """No decay at all, and decays whose products over a chunk leave float32."""
    check(150, [0, 150], 1, 2, 64, 64, dtype, g_scale=g_scale, seed=5)


def test_reset_by_minus_infinity():
    h = make(100, [0, 100], 1, 1, 32, 32, F32)
    h["g"][40] = -math.inf
    h["g"][70] = -3e38
    d = to_dev(h)
    o, s1, mags, kept = R.delta(*(h[n] for n in X), [0, 100], h["s0"], 32 ** -0.5)
    f = fwd(d)
    compare(f["o"], o, mags["o"], R.allowed(4), "o")
    want, mags = R.delta_bwd(h["do"], kept, h["ds1"], 1)
    r = bwd(d, f)
    for n in want:
        compare(r[n], want[n], mags[n], 2 * R.allowed(4), n)
    assert r["dg"][40].item() == 0.0 and r["dg"][70].item() == 0.0
    # a reset is the start of a sequence from zeros
    e = dict(d, offs=torch.tensor([0, 40, 100], dtype=torch.int32).cuda(), s0=torch.cat([d["s0"], torch.zeros_like(d["s0"])]),
             ds1=None)
    compare(fwd(e)["o"], o, mags_o(h, kept), R.allowed(4), "o")


def mags_o(h, kept):
    return (kept["q"].norm(dim=2).amax(0) * kept["most"][0] * 32 ** -0.5)[None, :, None].expand(h["v"].shape)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_beta_of_zero_and_two(dtype):
    h = make(130, [0, 130], 1, 2, 64, 64, dtype, seed=4)
    h["beta"][::3] = 0.0
    h["beta"][1::5] = 2.0
    o, s1, mags, kept = R.delta(*(h[n] for n in X), [0, 130], h["s0"], 0.125)
    d = to_dev(h)
    f = fwd(d)
    n = R.allowed(5)
    compare(f["o"], o, mags["o"], n, "o")
    want, mags = R.delta_bwd(h["do"], kept, h["ds1"], 2)
    for name, x in bwd(d, f).items():
        compare(x, want[name], mags[name], 2 * n, name)


def test_equal_keys():
    """One key throughout, beta of 1: the chunk's system is as far from the identity as unit keys make it."""
    h = make(128, [0, 128], 1, 1, 64, 64, F32, g_scale=0.0)
    h["k"][:] = h["k"][:1]
    h["beta"][:] = 1.0
    o, s1, mags, kept = R.delta(*(h[n] for n in X), [0, 128], h["s0"], 0.125)
    d = to_dev(h)
    f = fwd(d)
    compare(f["o"], o, mags["o"], R.allowed(4), "o")
    want, mags = R.delta_bwd(h["do"], kept, h["ds1"], 1)
    for name, x in bwd(d, f).items():
        compare(x, want[name], mags[name], 2 * R.allowed(4), name)


def test_nan_stays_in_its_sequence_and_head():
    h = make(200, [0, 90, 200], 2, 2, 32, 32, F32)
    d = to_dev(h)
    f = fwd(d)
    for name in ("q", "k", "v", "g", "beta"):
        e = {n: x.clone() if torch.is_tensor(x) else x for n, x in d.items()}
        e[name][30, 1] = math.nan
        o = fwd(e)["o"]
        assert torch.isnan(o[30, 1]).any(), name
        assert torch.equal(o[90:], f["o"][90:]) and torch.equal(o[:, 0], f["o"][:, 0]), name


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [2, 45])
def test_nan_outside_the_sequences_and_in_another(H, dtype):
    """What lies in front of, behind and in other sequences or heads changes no bit, in either form of the chains."""
    h = make(230, [7, 90, 200], H, H, 64, 48, dtype, seed=15)
    d = to_dev(h)
    f = fwd(d)
    r = bwd(d, f)
    e = {n: x.clone() if torch.is_tensor(x) else x for n, x in d.items()}
    for name in ("q", "k", "v", "g", "beta", "do"):
        e[name][:7] = math.nan
        e[name][200:] = math.inf
    f2 = fwd(e)
    r2 = bwd(e, f2)
    for x, y in zip([f["o"], f["s1"]] + list(r.values()), [f2["o"], f2["s1"]] + list(r2.values())):
        assert torch.equal(x, y)
    e["v"][40, 1] = math.nan
    e["do"][50, 1] = math.inf
    f2 = fwd(e)
    r2 = bwd(e, f2)
    assert torch.isnan(f2["o"][40:90, 1]).all() and torch.equal(f2["o"][90:], f["o"][90:]) and torch.equal(f2["o"][:, 0], f["o"][:, 0])
    assert torch.equal(f2["s1"][1], f["s1"][1]) and torch.equal(f2["s1"][0, 0], f["s1"][0, 0])
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        assert torch.equal(r2[n][90:], r[n][90:]) and torch.equal(r2[n][:, 0], r[n][:, 0]), n


def test_gradients_against_differences():
    """Central differences of sum(o do) + sum(s1 ds1) of the kernels along random directions. Their step's own error is
    what the float64 differences of the same step are off; each of the two values has rounding errors of at most
    2^-24 allowed() of its magnitude per output, independent of each other."""
    offs, sc = [0, 30, 70], 24 ** -0.5
    h = make(70, offs, 1, 2, 24, 20, F32, seed=9)
    d = to_dev(h)
    r = bwd(d, fwd(d))
    o, s1, mags, kept = R.delta(*(h[n] for n in X), offs, h["s0"], sc)
    exact, _ = R.delta_bwd(h["do"], kept, h["ds1"], 2)
    noise = 2.0 ** -24 * R.allowed(2) * math.hypot((mags["o"] * h["do"]).norm(), (mags["s1"] * h["ds1"]).norm())

    def on_gpu(e):
        f = fwd(e)
        return ((f["o"].double() * d["do"].double()).sum() + (f["s1"].double() * d["ds1"].double()).sum()).item()

    def in_64_bits(e):
        o, s1, _, _ = R.delta(*(e[n] for n in X), offs, e["s0"], sc)
        return ((o * h["do"].double()).sum() + (s1 * h["ds1"].double()).sum()).item()
    gen = torch.Generator().manual_seed(2)
    eps = 2.0 ** -7
    for name, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("g", "dg"), ("beta", "dbeta"), ("s0", "ds0")):
        u = torch.randn(h[name].shape, generator=gen)
        want = (exact[grad] * u.double()).sum().item()
        host = [in_64_bits(dict(h, **{name: h[name].double() + s * eps * u.double()})) for s in (1, -1)]
        off = abs((host[0] - host[1]) / (2 * eps) - want)
        assert off < 0.02 * abs(want) + 0.02, (name, off, want)
        # the float32 inputs of either side are rounded: half a step of each, through the gradient
        moved = 2.0 ** -24 * (exact[grad].abs() * (h[name].abs().double() + eps * u.abs().double())).norm().item() * 8
        up, dn = (on_gpu(dict(d, **{name: d[name] + s * eps * u.cuda()})) for s in (1, -1))
        got = (r[grad].cpu().double() * u.double()).sum().item()
        assert abs((up - dn) / (2 * eps) - got) <= 1.5 * off + (noise + moved) / eps, name


@pytest.mark.parametrize("dtype", [BF, F32])
def test_replay_under_load_with_poisoned_workspaces(dtype):
    h = make(700, [0, 300, 333, 690], 2, 4, 128, 128, dtype, seed=7)
    d = to_dev(h)
    load, first = SideLoad(64, 4), None
    need = (dg.det_delta_rule_workspace_size(700, 3, 2, 4, 128, 128, 0 if dtype == BF else 1),
            dg.det_delta_rule_bwd_workspace_size(700, 3, 2, 4, 128, 128, 0 if dtype == BF else 1))
    for i in range(8):
        load.kick()
        ws = [torch.full((n // 4,), (math.nan, 3e38, -1.0)[i % 3], device="cuda").view(torch.uint8) for n in need]
        f = fwd(d, ws=ws[0])
        r = bwd(d, f, ws=ws[1])
        chunks = sum(-(-n // (64 if dtype == BF else 32)) for n in (300, 33, 357))
        got = [f["o"], f["s1"], f["states"][:chunks], *r.values()]
        if first is None:
            first = [x.clone() for x in got]
        else:
            for a, b in zip(first, got):
                assert torch.equal(a, b)
        assert not torch.isnan(first[2]).any() and torch.isnan(f["states"][chunks:]).all()
    load.wait()


def test_bits_do_not_depend_on_other_sequences_or_heads():
    """Each sequence and head alone gives its rows of the packed call, though the launch shapes differ."""
    h = make(400, [0, 150, 400], 3, 3, 128, 128, BF, seed=8)
    d = to_dev(h)
    f = fwd(d)
    r = bwd(d, f)
    for s, (a, b) in enumerate(((0, 150), (150, 400))):
        for i in range(3):
            e = {n: x[a:b, i:i + 1].contiguous() for n, x in d.items() if n in X + ("do",)}
            e.update(offs=torch.tensor([0, b - a], dtype=torch.int32).cuda(), s0=d["s0"][s:s + 1, i:i + 1].contiguous(),
                     ds1=d["ds1"][s:s + 1, i:i + 1].contiguous())
            g = fwd(e)
            assert torch.equal(g["o"][:, 0], f["o"][a:b, i])
            q = bwd(e, g)
            for n in ("dq", "dk", "dv"):
                assert torch.equal(q[n][:, 0], r[n][a:b, i]), n
            assert torch.equal(q["dg"][:, 0], r["dg"][a:b, i]) and torch.equal(q["ds0"][0, 0], r["ds0"][s, i])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replays_and_two_streams(dtype):
    h = make(300, [0, 100, 300], 1, 2, 64, 64, dtype, seed=6)
    d = to_dev(h)
    f = fwd(d)
    want = [f["o"].clone(), f["s1"].clone()] + [x.clone() for x in bwd(d, f).values()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        fo, ro = fwd(d), None
        ro = bwd(d, fo)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        fwd(d, out=fo)
        bwd(d, fo, out=ro)
    for i in range(4):
        for x in [fo["o"], fo["s1"]] + list(ro.values()):
            x.fill_(float(i))
        g.replay()
        e = fwd(d)      # eager work between the replays
        torch.cuda.synchronize()
        assert torch.equal(e["o"], want[0])
        for a, b in zip([fo["o"], fo["s1"]] + list(ro.values()), want):
            assert torch.equal(a, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        x = fwd(d)
        y = bwd(d, x)
        torch.cuda.synchronize()
        outs.append((x, y))
    for s, (x, y) in zip(streams, outs):
        fwd(d, stream=s, out=x)
        bwd(d, x, stream=s, out=y)
    torch.cuda.synchronize()
    for x, y in outs:
        for a, b in zip([x["o"], x["s1"]] + list(y.values()), want):
            assert torch.equal(a, b)


# ------------------------------------------------------------------- single tokens
def step(d, state, slots=None, scale=None, stream=None):
    o = torch.full_like(d["v"], 7.0)
    dg.det_delta_rule_step(*(d[n] for n in X), state, o, slots=slots, scale=scale, stream=stream)
    return o


def check_step(B, N, slots, Hk, H, dk, dv, dtype, extra=0, seed=0, g=None):
    h = make(B, [0, B], Hk, H, dk, dv, dtype, seed=seed)
    if g is not None:
        h["g"][:] = g
    d = to_dev(h, extra)
    state = torch.randn(N, H, dk, dv, generator=torch.Generator().manual_seed(seed))
    want, o = state.double(), torch.zeros(B, H, dv).double()
    sl = list(range(B)) if slots is None else slots
    q, k = R._heads(h["q"], H), R._heads(h["k"], H)
    mag = torch.zeros(B, H, dv).double()
    for b, s in enumerate(sl):
        if not 0 <= s < N:
            continue
        kept = want[s] * h["g"][b].double().exp()[:, None, None]
        n = h["v"][b].double() - (k[b][:, :, None] * kept).sum(1)
        u = h["beta"][b].double()[:, None] * n
        want[s] = kept + k[b][:, :, None] * u[:, None, :]
        o[b] = dk ** -0.5 * (q[b][:, :, None] * want[s]).sum(1)
        um = h["beta"][b].double()[:, None] * (h["v"][b].double().abs() + (k[b].abs()[:, :, None] * kept.abs()).sum(1))
        mag[b] = dk ** -0.5 * ((q[b].abs()[:, :, None] * kept.abs()).sum(1) + (q[b] * k[b]).abs().sum(1, keepdim=True) * um)
    got = state.cuda()
    so = step(d, got, None if slots is None else torch.tensor(slots, dtype=torch.int32).cuda())
    # sums of dk terms (chains of at most 16 rows, at most 32 of them), the decay 4, u and the last products 6, for
    # every token that its state has taken
    n = (16 + 32 + 10) * max(1, max(sl.count(s) for s in sl)) if sl else 1
    R.assert_close(so, o, mag, n, "o")
    R.assert_close(got, want, (want.abs().amax(2, keepdim=True) + state.double().abs().amax(2, keepdim=True) + 4.0).expand_as(want),
                   n, "state")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dk,dv", [(1, 1), (3, 5), (64, 64), (128, 128), (127, 113), (33, 70), (128, 4), (5, 128)])
def test_step_sizes(dk, dv, dtype):
    check_step(5, 9, [3, 8, 0, 1, 5], 2, 4, dk, dv, dtype, seed=dk)


@pytest.mark.parametrize("B,H,dv", [(1, 1, 128), (200, 3, 128), (130, 4, 128), (70, 8, 64), (300, 2, 30)])
def test_step_launch_shapes(B, H, dv):
    check_step(B, B + 3, None, 1, H, 40, dv, BF, seed=B)


def test_step_padding_and_repeated_slots():
    check_step(12, 4, [2, -1, 2, 0, 4, 2, 100, 0, -7, 3, 2, 0], 1, 2, 48, 50, F32)
    check_step(300, 3, [i % 5 - 1 for i in range(300)], 1, 1, 16, 16, F32, seed=2)
    check_step(4, 1, [0, 0, 0, 0], 1, 2, 64, 64, BF, seed=3)


def test_step_strides_and_decays():
    check_step(6, 6, None, 2, 2, 64, 65, BF, extra=3)
    check_step(6, 6, None, 2, 2, 64, 64, F32, g=0.0)
    check_step(6, 6, None, 2, 2, 64, 64, F32, g=-math.inf)


def test_step_leaves_other_states_alone_and_replays():
    h = make(6, [0, 6], 1, 4, 128, 128, BF)
    d = to_dev(h)
    slots = torch.tensor([7, -1, 2, 9, 2, 30], dtype=torch.int32).cuda()
    state0 = torch.randn(12, 4, 128, 128, device="cuda")
    s1 = state0.clone()
    o = step(d, s1, slots)
    touched = torch.zeros(12, dtype=torch.bool)
    touched[[7, 2, 9]] = True
    for i in range(12):
        assert torch.equal(s1[i], state0[i]) != bool(touched[i]), i
    assert (o[1] == 0).all() and (o[5] == 0).all()
    g, s2, o2 = torch.cuda.CUDAGraph(), state0.clone(), torch.zeros_like(o)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    dg.det_delta_rule_step(*(d[n] for n in X), s2, o2, slots=slots, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(s2, s1) and torch.equal(o2, o)
    with torch.cuda.graph(g):
        dg.det_delta_rule_step(*(d[n] for n in X), s2, o2, slots=slots)
    want = state0.clone()
    s2.copy_(state0)
    for _ in range(3):
        g.replay()
        e = step(d, want, slots)
        torch.cuda.synchronize()
        assert torch.equal(s2, want) and torch.equal(o2, e)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_then_tokens_is_one_longer_prefill(dtype):
    """A prompt's final state goes into a cache slot, five tokens follow one by one."""
    h = make(75, [0, 75], 2, 4, 64, 96, dtype, seed=11)
    d = to_dev(h)
    o, s1, mags, _ = R.delta(*(h[n] for n in X), [0, 75], h["s0"], 0.125)
    cut = dict({n: d[n][:70] for n in X}, offs=torch.tensor([0, 70], dtype=torch.int32).cuda(), s0=d["s0"])
    cache = torch.zeros(3, 4, 64, 96, device="cuda")
    f = fwd(cut, 0.125, states=False)
    cache[1] = f["s1"][0]
    slots = torch.tensor([1], dtype=torch.int32).cuda()
    n = R.allowed(8)
    for t in range(70, 75):
        e = {m: d[m][t:t + 1] for m in X}
        compare(step(e, cache, slots, 0.125), o[t:t + 1], mags["o"][t:t + 1], n, "o")
    compare(cache[1:2], s1, mags["s1"], n, "state")
