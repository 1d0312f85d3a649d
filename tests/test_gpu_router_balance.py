"""det_router_balance and its backward against float64, with the shapes, strides,
offsets and masks where they can go wrong; run-to-run bits; graphs; streams."""
import math

import numpy as np
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64
from tests.gpu_util import SideLoad, note

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, E, K, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * spread).to(dtype)
    ids = torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    ids[torch.rand(T, K, generator=g) < 0.05] = -1
    return z, ids


def strided(t, ld, shift):
    """t on the GPU with row stride ld (>= its width), starting `shift` elements into an allocation."""
    rows, cols = t.shape
    buf = torch.full((shift + max(rows, 1) * ld,), 77, dtype=t.dtype, device="cuda")
    v = buf[shift:shift + rows * ld].view(rows, ld)[:, :cols] if rows else buf[:0].view(0, ld)[:, :cols]
    v.copy_(t)
    return v


def fwd(z, ids, offs, coeff=0.01, score="softmax", ws=None, stream=None):
    S, E = offs.numel() - 1, z.shape[1]
    counts = torch.full((S, E), -7, dtype=torch.int32, device="cuda")
    psum = torch.full((S, E), math.nan, device="cuda")
    loss = torch.full((S,), math.nan, device="cuda")
    dg.det_router_balance(z, ids, offs, counts, psum, loss, coeff=coeff, score=score, ws=ws, stream=stream)
    return loss, counts, psum


def roundings(z, E, T):
    """Roundings on the way to p and P: the exponent's (its arguments reach the row's spread R: the difference, and
    for the sigmoid score the two logarithms, 3 R + 8), exp's 3 in numerator and denominator, the row sum's chain of
    16 and tree of 6, the quotient's 2; then P's chain of a lane (at most T / 16 rows) and its tree of 14."""
    fin = z.double()[torch.isfinite(z.double())]
    R = float(fin.max() - fin.min()) + float(fin.abs().max()) if fin.numel() else 0.0
    return 3 * R + 8 + 6 + 16 + 6 + 2 + min(T, 16 + T / 16) + 14


def offsets(*o):
    return torch.tensor(o, dtype=torch.int32, device="cuda")


def check(T, E, K, dtype, offs, score, seed=0, ld=None, shift=0, z=None, coeff=0.01):
    z0, ids = make(T, E, K, dtype, seed)
    z = z0 if z is None else z
    zd = strided(z, ld or E, shift)
    idd = strided(ids, K + (3 if ld else 0), shift)
    od = offsets(*offs)
    loss, counts, psum = fwd(zd, idd, od, coeff, score)
    wl, wc, wp = ref64.router(z, ids, offs, coeff, score)
    assert torch.equal(counts.cpu(), wc)
    n = roundings(z, E, T)
    ref64.assert_close(psum, wp, wp.nan_to_num(), n, "prob_sum")
    ref64.assert_close(loss, wl, wl.nan_to_num(), n + 4, "loss")
    # backward, into an output with its own stride and old contents
    g = torch.Generator().manual_seed(seed + 1)
    dloss = torch.rand(len(offs) - 1, generator=g) * 100 + 1
    old = torch.randn(T, E, generator=g).to(dtype)
    dz = strided(old, (ld or E) + 5, shift)
    dg.det_router_balance_bwd(dz, zd, od, counts, dloss.cuda(), K, coeff=coeff, score=score)
    wd, wm = ref64.router_bwd(z, offs, wc, dloss, K, coeff, score, old)
    ref64.assert_close(dz, wd, wm.nan_to_num(), n + 30, "dlogits")
    b = ref64.bounds(offs, T)
    assert torch.equal(dz.cpu()[:b[0]], old[:b[0]]) and torch.equal(dz.cpu()[b[-1]:], old[b[-1]:])
    if ld:  # the gaps between the rows keep their fill
        gap = dz._base if dz._base is not None else dz
        flat = gap.flatten()[shift:shift + T * (ld + 5)].view(T, ld + 5)[:, E:]
        assert bool((flat == 77).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 8, 2), (7, 3, 2), (33, 16, 4), (100, 31, 1), (257, 64, 6),
                                   (64, 65, 8), (301, 128, 4), (129, 200, 3), (515, 256, 8), (90, 511, 5),
                                   (70, 512, 2), (40, 513, 2), (35, 1000, 7), (9, 1024, 16), (3000, 17, 2), (8300, 16, 2), (700, 250, 3), (500, 500, 2),
                                   (300, 700, 4), (2100, 72, 2), (17000, 8, 1), (1300, 128, 2), (4200, 32, 1)])
def test_sizes(T, E, K, dtype, score):
    check(T, E, K, dtype, [0, T], score, seed=T + E)


@pytest.mark.parametrize("offs", [[0, 0, 5, 5, 60, 97], [10, 50], [3, 20, 20, 90], [-5, 40, 1000], [60, 20, 80],
                                  [0, 0], [97, 97], [200, 300], [0] * 130 + [97]])
@pytest.mark.parametrize("E", [5, 64])
def test_segments_empty_outside_and_unordered(offs, E):
    """Empty segments, tokens before the first and behind the last, offsets outside [0, T] and decreasing ones."""
    check(97, E, 3, F32, offs, "softmax", seed=len(offs))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,ld,shift", [(64, 71, 1), (10, 13, 3), (257, 300, 5), (64, 64, 1)])
def test_strides_and_unaligned_rows(E, ld, shift, dtype):
    check(77, E, 4, dtype, [1, 30, 75], "sigmoid", seed=9, ld=ld, shift=shift)


def test_many_segments():
    g = torch.Generator().manual_seed(3)
    cuts = torch.randint(0, 2001, (700,), generator=g).sort().values.tolist()
    check(2000, 24, 2, BF, [0] + cuts + [2000], "softmax", seed=4)
    check(700, 400, 2, F32, [0] * 650 + list(range(0, 700, 2)) + [700], "softmax", seed=5)   # tiles of several workgroups


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_rows(score):
    """-inf logits (an expert switched off), rows of nothing but -inf (p = 0), the type's lowest value."""
    z, _ = make(50, 40, 2, F32, 1)
    z[:, 7] = -math.inf
    z[5] = -math.inf
    z[6, :39] = -math.inf
    z[8, :20] = torch.finfo(F32).min
    z[9] = torch.finfo(F32).min
    zd, od = z.cuda(), offsets(0, 50)
    ids = torch.zeros(50, 2, dtype=torch.int32)
    loss, counts, psum = fwd(zd, ids.cuda(), od, score=score)
    wl, wc, wp = ref64.router(z, ids, [0, 50], 0.01, score)
    ref64.assert_close(psum, wp, wp, 120, "prob_sum")
    assert torch.equal(counts.cpu(), wc) and int(wc[0, 0]) == 100
    dz = torch.full_like(zd, 3.0)
    dg.det_router_balance_bwd(dz, zd, od, counts, torch.ones(1, device="cuda"), 2, coeff=0.01, score=score)
    assert bool(torch.isfinite(dz).all()) and bool((dz[5] == 0).all())
    # expert 7 is masked in every row but row 9, whose 40 equal logits give it p = 1 / 40
    assert bool((dz[:9, 7] == 0).all()) and bool((dz[10:, 7] == 0).all())
    wd, wm = ref64.router_bwd(z, [0, 50], wc, torch.ones(1), 2, 0.01, score, torch.zeros(50, 40))
    ref64.assert_close(dz, wd, wm, 150, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E", [7, 24, 300])
def test_rows_of_very_negative_logits(score, E):
    """Rows whose sigmoids underflow (-150 and below) keep their ratios, beside ordinary rows of the same wave."""
    z, _ = make(40, E, 2, F32, 3)
    z[::3] -= 150.0
    z[1::6] -= 1000.0
    z[5, 0] = -40.0
    check(40, E, 2, F32, [0, 13, 40], score, z=z)


def test_nan_and_infinity_stay_in_their_row_and_outside_rows_are_not_read():
    z, ids = make(60, 24, 2, F32, 2)
    z[0] = math.nan          # before the first segment
    z[59, 3] = math.inf      # behind the last
    od = offsets(1, 30, 59)
    clean = fwd(z.cuda(), ids.cuda(), od)
    assert all(bool(torch.isfinite(t.float()).all()) for t in clean)
    z[40, 2] = math.nan
    z[41, 1] = math.inf
    z[42] = math.nan
    loss, counts, psum = fwd(z.cuda(), ids.cuda(), od)
    assert torch.equal(loss[0], clean[0][0]) and torch.equal(psum[0], clean[2][0]) and torch.equal(counts, clean[1])
    assert bool(torch.isnan(psum[1]).all()) and bool(torch.isnan(loss[1]))
    dz = torch.zeros_like(z).cuda()
    dg.det_router_balance_bwd(dz, z.cuda(), od, counts, torch.ones(2, device="cuda"), 2)
    bad = torch.isnan(dz).any(1).nonzero().flatten().tolist()
    assert bad == [40, 41, 42] and bool(torch.isnan(dz[40]).all())


def test_ids_outside_and_repeated():
    z, _ = make(20, 6, 3, F32, 5)
    ids = torch.tensor([[2, 2, 2], [-1, 6, 5], [2 ** 31 - 1, -2 ** 31, 0]], dtype=torch.int32).repeat(7, 1)[:20]
    _, counts, _ = fwd(z.cuda(), ids.cuda(), offsets(0, 20))
    assert counts.cpu()[0].tolist() == [6, 0, 21, 0, 0, 7]


def test_no_tokens_and_no_segments():
    z, ids = torch.zeros(0, 8, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    loss, counts, psum = fwd(z, ids, offsets(0, 0, 0))
    assert loss.tolist() == [0, 0] and int(counts.abs().sum()) == 0 and float(psum.abs().sum()) == 0
    loss, _, _ = fwd(torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), offsets(0))
    assert loss.numel() == 0
    dz = torch.ones(4, 8, device="cuda")
    dg.det_router_balance_bwd(dz, torch.zeros(4, 8, device="cuda"), offsets(0),
                              torch.zeros(0, 8, dtype=torch.int32, device="cuda"), torch.zeros(0, device="cuda"), 2)
    assert bool((dz == 1).all())


def test_gradient_against_differences():
    """The gradient of sum dloss * loss with the counts held, against central differences in float64."""
    for score in ("softmax", "sigmoid"):
        z, ids = make(6, 5, 2, F32, 11, spread=1.0)
        offs, dl = [0, 4, 6], torch.tensor([1.5, -0.5])
        _, counts, _ = ref64.router(z, ids, offs, 0.3, score)

        def total(zz):
            p = ref64.router_probs(zz, score)
            out = 0.0
            for s in range(2):
                n = offs[s + 1] - offs[s]
                P = p[offs[s]:offs[s + 1]].sum(0)
                out += float(dl[s]) * 0.3 * 5 / (2 * n * n) * float((counts[s].double() * P).sum())
            return out
        dz = torch.zeros(6, 5, device="cuda")
        dg.det_router_balance_bwd(dz, z.cuda(), offsets(*offs), counts.cuda(), dl.cuda(), 2, coeff=0.3, score=score)
        h = 1e-5
        for t in range(6):
            for e in range(5):
                a, b = z.double().clone(), z.double().clone()
                a[t, e] += h
                b[t, e] -= h
                num = (total(a) - total(b)) / (2 * h)   # error of order h^2 = 1e-10
                assert abs(num - float(dz[t, e])) < 1e-6, (score, t, e)


def test_summed_counts_of_two_ranks():
    """The backward takes counts other than the call's own (data-parallel sums), far from K N / E."""
    z, _ = make(40, 32, 2, F32, 6)
    counts = torch.randint(0, 2 ** 30, (1, 32), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    dz = torch.zeros(40, 32, device="cuda")
    dg.det_router_balance_bwd(dz, z.cuda(), offsets(0, 40), counts.cuda(), torch.ones(1, device="cuda"), 2, coeff=1.0)
    wd, wm = ref64.router_bwd(z, [0, 40], counts, torch.ones(1), 2, 1.0, "softmax", torch.zeros(40, 32))
    ref64.assert_close(dz, wd, wm, 120, "dlogits")


def test_rows_past_32_bit_offsets():
    """Row 2 of a logits view starts past 2^31 elements (2^32 bytes)."""
    ld = (1 << 30) + 8
    buf = torch.empty(2 * ld + 64, dtype=BF, device="cuda")
    z = buf.as_strided((3, 64), (ld, 1))
    src, ids = make(3, 64, 2, BF, 8)
    z.copy_(src)
    loss, counts, psum = fwd(z, ids.cuda(), offsets(0, 3))
    want = ref64.router(src, ids, [0, 3], 0.01, "softmax")
    ref64.assert_close(psum, want[2], want[2], roundings(src, 64, 3), "prob_sum")
    dz = torch.empty(2 * ld + 64, dtype=BF, device="cuda").as_strided((3, 64), (ld, 1))
    dg.det_router_balance_bwd(dz, z, offsets(0, 3), counts, torch.ones(1, device="cuda"), 2, coeff=0.01)
    wd, wm = ref64.router_bwd(src, [0, 3], want[1], torch.ones(1), 2, 0.01, "softmax", torch.zeros(3, 64))
    ref64.assert_close(dz, wd, wm, roundings(src, 64, 3) + 30, "dlogits")


def test_replay_under_load_with_poisoned_workspaces():
    z, ids = make(5000, 96, 4, BF, 12)
    z, ids, od = z.cuda(), ids.cuda(), offsets(0, 700, 2900, 4990)
    n = dg.det_router_balance_workspace_size(5000, 96, 4, 3)
    assert n > 0
    first, load = None, SideLoad(mib=64, iters=4)
    for fill in (0, 255, 127, 1, 255, 3, 0, 90):
        ws = torch.full((n + 256,), fill, dtype=torch.uint8, device="cuda")
        ws = ws[-ws.data_ptr() % 256:][:n]
        load.kick()
        out = fwd(z, ids, od, ws=ws)
        dz = torch.zeros_like(z)
        dg.det_router_balance_bwd(dz, z, od, out[1], torch.ones(3, device="cuda"), 4)
        got = [t.clone() for t in (*out, dz)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        assert bool((ws[:256] == fill).all())     # the header is left alone
    load.wait()
    note("router balance: 8 runs under load with poisoned workspaces, same bits")


def test_graph_replays_and_two_streams():
    z, ids = make(3000, 40, 2, BF, 13)
    z, ids, od = z.cuda(), ids.cuda(), offsets(0, 1000, 3000)
    counts = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
    psum, loss, dz = torch.zeros(2, 40, device="cuda"), torch.zeros(2, device="cuda"), torch.zeros_like(z)
    one = torch.ones(2, device="cuda")

    def step():
        dg.det_router_balance(z, ids, od, counts, psum, loss, coeff=0.5)
        dg.det_router_balance_bwd(dz, z, od, counts, one, 2, coeff=0.5)
    graphs = []
    for _ in range(2):      # two graphs, each with a workspace of its own
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for r in range(4):
        z.mul_(0.9)
        step()
        want = [t.clone() for t in (loss, counts, psum, dz)]
        for g in graphs:
            for t in (loss, psum, dz):
                t.fill_(7)
            counts.fill_(7)
            torch.empty(1 << 20, device="cuda").normal_()    # eager work between the replays
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((loss, counts, psum, dz), want)), r
    # the same call on two streams at once, through the stream argument, without a workspace from the caller
    want = [t.clone() for t in fwd(z, ids, od, 0.5)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for r in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                bufs = (torch.zeros(2, device="cuda"), torch.zeros_like(counts), torch.zeros_like(psum))
            dg.det_router_balance(z, ids, od, bufs[1], bufs[2], bufs[0], coeff=0.5, stream=s)
            outs.append(bufs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


def test_a_tensor_on_the_host_is_refused():
    z, ids = make(8, 6, 2, F32, 1)
    with pytest.raises(ValueError, match="ids"):
        fwd(z.cuda(), ids, offsets(0, 8))
    with pytest.raises(ValueError, match="offs"):
        fwd(z.cuda(), ids.cuda(), torch.tensor([0, 8], dtype=torch.int32))
    small = torch.zeros(64, dtype=torch.uint8, device="cuda")
    big, big_ids = make(20000, 32, 2, F32, 1)
    with pytest.raises(dg.DetError, match="workspace"):
        fwd(big.cuda(), big_ids.cuda(), offsets(0, 20000), ws=small)
    with pytest.raises(ValueError, match="workspace"):
        fwd(big.cuda(), big_ids.cuda(), offsets(0, 20000), ws=small.cpu())
