"""det_topk_distill and its backward against float64, with the shapes, strides,
ids and masks where they can go wrong; run-to-run bits; graphs; streams."""
import math

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64
from tests.gpu_util import SideLoad, note
from tests.test_gpu_router_balance import strided

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def make(T, V, K, dtype, t_dtype, seed):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, V, generator=g) * 3).to(dtype)
    ids = torch.randint(0, V, (T, K), generator=g, dtype=torch.int32)     # repeated ids happen
    ids[torch.rand(T, K, generator=g) < 0.1] = -1
    t = (torch.randn(T, K, generator=g) * 3).to(t_dtype)
    dloss = torch.randn(T, generator=g)
    if T > 2:
        ids[1] = -1         # a token without a teacher
        dloss[2] = 0.0
    return z, ids, t, dloss


def fwd(z, ids, t, tau=1.0, ws=None, stream=None):
    loss = torch.full((z.shape[0],), 55.0, device="cuda")
    lse = torch.full((z.shape[0],), 55.0, device="cuda")
    dg.det_topk_distill(z, ids, t, loss, lse, tau=tau, ws=ws, stream=stream)
    return loss, lse


def roundings(z, t, tau, V):
    """Exponents: at most R = the largest |z| / tau plus the largest |lse| (two products and a difference: 3 R);
    exp's 3; the sums' chains: 16 + 8 in a lane's step, V / 8192 + 8 steps, trees of 6 + 4, the join of pieces
    with a factor each (3 x 8); logarithm and scale 4; the teacher's softmax the same with its chain of 16 + 6."""
    r = float(z.double()[torch.isfinite(z.double())].abs().max()) / tau if z.numel() else 0.0
    rt = float(t.double()[torch.isfinite(t.double())].abs().max()) / tau if t.numel() else 0.0
    return 3 * (2 * r + math.log(max(V, 2))) + 6 * rt + 3 + 24 + V / 8192 + 8 + 10 + 24 + 4 + 3 + 22


def check(T, V, K, dtype, t_dtype=F32, tau=1.0, seed=0, ld=None, shift=0, data=None):
    z, ids, t, dloss = data or make(T, V, K, dtype, t_dtype, seed)
    zd = strided(z, ld or V, shift)
    idd, td = strided(ids, K + (3 if ld else 0), shift), strided(t, K + (5 if ld else 0), shift)
    loss, lse = fwd(zd, idd, td, tau)
    wl, wm, ws = ref64.distill(z, ids, t, tau)
    n = roundings(z, t, tau, V)
    ref64.assert_close(lse, ws, torch.ones_like(ws) + 0.1 * ws.abs().nan_to_num(posinf=0.0, neginf=0.0), n, "lse")
    ref64.assert_close(loss, wl, wm.nan_to_num(posinf=0.0) + 1.0, n, "loss")
    old = torch.full((T, V), 9.0).to(dtype)
    dz = strided(old, (ld or V) + 7, shift)
    dg.det_topk_distill_bwd(dz, zd, idd, td, lse, dloss.cuda(), tau=tau)
    wd, wdm = ref64.distill_bwd(z, ids, t, lse.cpu(), dloss, tau)
    ref64.assert_close(dz, wd, wdm.nan_to_num(), n, "dlogits")
    if T > 2 and data is None:
        assert float(loss[1]) == 0 and bool((dz[1:3] == 0).all())
    if ld:
        flat = dz._base.flatten()[shift:shift + T * (ld + 7)].view(T, ld + 7)[:, V:]
        assert bool((flat == 77).all())


@pytest.mark.parametrize("dtype,t_dtype", [(BF, F32), (F32, BF)])
@pytest.mark.parametrize("T,V,K", [(1, 1, 1), (3, 2, 1), (4, 7, 3), (5, 8, 16), (9, 255, 8), (6, 2047, 64),
                                   (7, 2048, 65), (3, 8192, 5), (4, 8193, 130), (5, 16385, 1024), (2, 50001, 33), (2, 262145, 40), (3, 600001, 7), (600, 3001, 9), (513, 1000, 300), (520, 66001, 5), (516, 131101, 3),
                                   (1, 131072, 1), (1030, 300, 4)])
def test_sizes(T, V, K, dtype, t_dtype):
    check(T, V, K, dtype, t_dtype, tau=1.0 if T % 2 else 2.5, seed=T * 7 + V)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,ld,shift", [(1001, 1001, 1), (1001, 1013, 3), (20000, 20001, 7), (20001, 20001, 0),
                                        (8200, 8201, 5), (16450, 16451, 33)])
def test_strides_and_unaligned_rows(V, ld, shift, dtype):
    check(6, V, 20, dtype, dtype, tau=0.7, seed=2, ld=ld, shift=shift)


@pytest.mark.parametrize("tau", [0.05, 1.0, 30.0])
def test_temperature(tau):
    check(8, 5000, 12, F32, tau=tau, seed=3)


def test_no_slots_and_no_tokens():
    z = torch.randn(3, 100, device="cuda")
    ids, t = torch.zeros(3, 0, dtype=torch.int32, device="cuda"), torch.zeros(3, 0, device="cuda")
    loss, lse = fwd(z, ids, t)
    assert loss.tolist() == [0, 0, 0]
    assert torch.allclose(lse.double(), torch.logsumexp(z.double(), 1), rtol=0, atol=1e-5)
    dz = torch.ones_like(z)
    dg.det_topk_distill_bwd(dz, z, ids, t, lse, torch.ones(3, device="cuda"))
    assert bool((dz == 0).all())
    e = torch.zeros(0, device="cuda")
    dg.det_topk_distill(z[:0], ids[:0], t[:0], e, e.clone())
    dg.det_topk_distill_bwd(z[:0].clone(), z[:0], ids[:0], t[:0], e, e)


def test_the_same_word_in_many_slots():
    V = 3000
    z, ids, t, dl = make(5, V, 96, F32, F32, 4)
    ids[0] = 17
    ids[3, :50] = 2999
    ids[4, ::2] = 0
    check(5, V, 96, F32, data=(z, ids, t, dl), seed=4)


def test_ids_outside_and_nan_in_unused_slots():
    z, ids, t, dl = make(6, 500, 12, F32, F32, 5)
    ids[0, :4] = torch.tensor([500, -2, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    t[0, :4] = torch.tensor([math.nan, math.inf, math.nan, -math.inf])
    t[1] = math.nan            # the token without a teacher
    check(6, 500, 12, F32, data=(z, ids, t, dl))


def test_masked_words_and_teacher_slots():
    """-inf and the type's lowest value in student and teacher logits; a teacher of -inf only; a teacher word that the
    student has masked (an infinite loss, a finite gradient)."""
    low = torch.finfo(F32).min
    z, ids, t, dl = make(8, 9000, 10, F32, F32, 6)
    ids = torch.stack([torch.randperm(9000, generator=torch.Generator().manual_seed(i))[:10] for i in range(8)]).int()
    z[:, 5000:] = -math.inf
    z[:, 4000:5000] = low
    ids = ids.clamp(max=3999)
    t[0, 3:] = -math.inf
    t[4] = -math.inf
    t[5, :5] = low
    z[6, :] = -math.inf
    z[6, 8999] = 1.0           # one word left, at the end
    ids[6] = 8999
    ids[7, 0] = 8000           # masked by the student
    zd, idd, td = z.cuda(), ids.cuda(), t.cuda()
    loss, lse = fwd(zd, idd, td)
    wl, wm, ws = ref64.distill(z, ids, t, 1.0)
    ref64.assert_close(lse, ws, ws.abs() + 1, 300, "lse")
    ref64.assert_close(loss, wl, wm.nan_to_num(posinf=0.0) + 1, 300, "loss")
    assert float(loss[4]) == 0 and math.isinf(float(loss[7]))
    dz = torch.full_like(zd, 5.0)
    dl = torch.ones(8)
    dg.det_topk_distill_bwd(dz, zd, idd, td, lse, dl.cuda())
    wd, wdm = ref64.distill_bwd(z, ids, t, lse.cpu(), dl, 1.0)
    assert bool(torch.isfinite(dz).all())
    ref64.assert_close(dz, wd, wdm, 300, "dlogits")


def test_nan_stays_in_its_row_and_a_zero_weight_clears_it():
    z, ids, t, _ = make(6, 3000, 8, F32, F32, 7)
    ids = ids.clamp(min=0)
    z[2, 100] = math.nan
    z[3, 7] = math.nan
    loss, lse = fwd(z.cuda(), ids.cuda(), t.cuda())
    assert torch.isnan(loss).nonzero().flatten().tolist() == [2, 3]
    w = torch.ones(6, device="cuda")
    w[3] = 0.0
    dz = torch.full((6, 3000), 5.0, device="cuda")
    dg.det_topk_distill_bwd(dz, z.cuda(), ids.cuda(), t.cuda(), lse, w)
    assert torch.isnan(dz).any(1).nonzero().flatten().tolist() == [2] and bool((dz[3] == 0).all())


def test_gradient_against_differences():
    z, ids, t, dl = make(4, 11, 3, F32, F32, 8)
    ids[0] = torch.tensor([4, 4, 9], dtype=torch.int32)
    tau, h = 1.7, 1e-5
    loss, lse = fwd(z.cuda(), ids.cuda(), t.cuda(), tau)
    dz = torch.zeros(4, 11, device="cuda")
    dg.det_topk_distill_bwd(dz, z.cuda(), ids.cuda(), t.cuda(), lse, dl.cuda(), tau=tau)
    for r in range(4):
        for v in range(11):
            a, b = z.double().clone(), z.double().clone()
            a[r, v] += h
            b[r, v] -= h
            num = float(dl[r]) * float(ref64.distill(a, ids, t, tau)[0][r] - ref64.distill(b, ids, t, tau)[0][r]) / (2 * h)
            assert abs(num - float(dz[r, v])) < 2e-6, (r, v)


def test_rows_past_32_bit_offsets():
    ld = (1 << 30) + 8
    V = 10001
    z = torch.empty(2 * ld + V, dtype=BF, device="cuda").as_strided((3, V), (ld, 1))
    dz = torch.empty(2 * ld + V, dtype=BF, device="cuda").as_strided((3, V), (ld, 1))
    src, ids, t, dl = make(3, V, 16, BF, F32, 9)
    ids[1], dl[2] = ids[0], 1.0
    z.copy_(src)
    loss, lse = fwd(z, ids.cuda(), t.cuda())
    dg.det_topk_distill_bwd(dz, z, ids.cuda(), t.cuda(), lse, dl.cuda())
    n = roundings(src, t, 1.0, V)
    wl, wm, ws = ref64.distill(src, ids, t, 1.0)
    ref64.assert_close(loss, wl, wm + 1, n, "loss")
    wd, wdm = ref64.distill_bwd(src, ids, t, lse.cpu(), dl, 1.0)
    ref64.assert_close(dz, wd, wdm, n, "dlogits")


@pytest.mark.parametrize("dtype,T,V", [(BF, 1030, 131072), (F32, 700, 100003)])
def test_gradients_past_the_caches(dtype, T, V):
    """A gradient larger than the last-level cache is stored another way: every row has the bits of a small call."""
    assert T * V * torch.finfo(dtype).bits // 8 >= 256 << 20
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(T, V, device="cuda", dtype=dtype, generator=g)
    ids = torch.randint(-1, V, (T, 40), device="cuda", dtype=torch.int32, generator=g)
    t, dl = torch.randn(T, 40, device="cuda", generator=g), torch.randn(T, device="cuda", generator=g)
    lse = torch.logsumexp(z.float(), 1)
    dz = torch.full_like(z, 9.0)
    dg.det_topk_distill_bwd(dz, z, ids, t, lse, dl)
    for r in range(0, T, 101):
        part = torch.full_like(z[r:r + 7], 5.0)
        n = part.shape[0]
        dg.det_topk_distill_bwd(part, z[r:r + 7], ids[r:r + 7], t[r:r + 7], lse[r:r + 7].contiguous(),
                                dl[r:r + 7].contiguous())
        assert torch.equal(dz[r:r + n], part), r


@pytest.mark.parametrize("T", [3, 1100])
def test_replay_under_load_with_poisoned_workspaces(T):
    V = 700001 if T == 3 else 3000
    z, ids, t, dl = [x.cuda() for x in make(T, V, 24, BF, F32, 10)]
    n = dg.det_topk_distill_workspace_size(T, V, 24)
    assert (n > 0) == (T == 3)
    first, load = None, SideLoad(mib=64, iters=4)
    for fill in (0, 255, 127, 1, 255, 3, 0, 90):
        ws = torch.full((n + 512,), fill, dtype=torch.uint8, device="cuda")
        ws = ws[-ws.data_ptr() % 256:][:n + 256]
        load.kick()
        out = fwd(z, ids, t, ws=ws)
        dz = torch.full_like(z, fill)
        dg.det_topk_distill_bwd(dz, z, ids, t, out[1], dl)
        got = [x.clone() for x in (*out, dz)]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
        assert bool((ws[:256] == fill).all())
    load.wait()
    note("distillation: 8 runs under load with poisoned workspaces, same bits")


def test_graph_replays_and_two_streams():
    z, ids, t, dl = [x.cuda() for x in make(6, 300001, 24, BF, F32, 11)]
    loss, lse, dz = torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda"), torch.zeros_like(z)

    def step():
        dg.det_topk_distill(z, ids, t, loss, lse, tau=2.0)
        dg.det_topk_distill_bwd(dz, z, ids, t, lse, dl, tau=2.0)
    graphs = []
    for _ in range(2):
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for r in range(4):
        z.mul_(0.9)
        step()
        want = [x.clone() for x in (loss, lse, dz)]
        for g in graphs:
            for x in (loss, lse, dz):
                x.fill_(7)
            torch.empty(1 << 20, device="cuda").normal_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip((loss, lse, dz), want)), r
    want = [x.clone() for x in fwd(z, ids, t)]
    torch.cuda.synchronize()
    outs = []
    for r in range(4):
        for s in [torch.cuda.Stream() for _ in range(2)]:
            with torch.cuda.stream(s):
                bufs = (torch.zeros(6, device="cuda"), torch.zeros(6, device="cuda"))
            dg.det_topk_distill(z, ids, t, *bufs, stream=s)
            outs.append(bufs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
