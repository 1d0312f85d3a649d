"""det_topk_distill and its backward on rows with logits far from 0 (the type's lowest
value, -1e30, -1e10 and the like): masked words in front of ordinary ones, rows that a
mask left empty, and rows that leave float32 once they are divided by the temperature."""
import math

import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64
from tests.test_gpu_topk_distill import fwd, roundings

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def reference(z, ids, t, dloss, tau):
    """(loss, its magnitude, lse, dlogits, its magnitude) in float64 from differences to the row's largest logit."""
    zd = z.double()
    top = zd.max(1, keepdim=True).values
    x = (zd - top) / tau
    logs = torch.logsumexp(x, 1, keepdim=True)
    lp = x - logs
    td = t.double()
    lq = torch.log_softmax((td - td.max(1, keepdim=True).values) / tau, 1)
    q = lq.exp()
    lpk = lp.gather(1, ids.long())
    loss = torch.where(q == 0, torch.zeros_like(q), q * (lq - lpk)).sum(1)
    mag = torch.where(q == 0, torch.zeros_like(q), q * (lq.abs() + lpk.abs())).sum(1)
    y = torch.zeros_like(zd).scatter_add(1, ids.long(), q)
    a = (dloss.double() / tau)[:, None]
    return loss, mag, (top / tau + logs)[:, 0], a * (lp.exp() - y), a.abs() * (lp.exp() + y)


def rows(V, K, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    fi = torch.finfo(dtype)
    z = torch.full((9, V), fi.min).to(dtype)              # 0, 1: nothing but the lowest value
    z[2, V // 3:] = -math.inf                             # 2: the lowest value and -inf
    z[3] = fi.max                                         # 3: the largest value everywhere
    z[4] = (torch.randn(V, generator=g) * 3).to(dtype)    # 4: ordinary words before masked ones
    z[4, V // 2:] = fi.min
    z[5] = fi.min / 2                                     # 5: half the lowest
    z[6] = z[4].flip(0)                                   # 6: ordinary words behind masked ones
    z[7] = -1e10                                          # 7: a smaller mask, everywhere
    z[8, :V // 2] = -1e30                                 # 8: and one of that kind in front of ordinary words
    z[8, V // 2:] = z[4, :V - V // 2].clamp(min=-20)
    ids = torch.stack([torch.randperm(V // 3, generator=g)[:K] for _ in range(9)]).int()
    ids[6] += V - V // 3
    ids[8] += V // 2
    t = torch.randn(9, K, generator=g) * 3
    t[1] = torch.finfo(F32).min                           # a teacher of nothing but the lowest value: equal weights
    return z, ids, t, torch.randn(9, generator=g) + 3


@pytest.mark.parametrize("tau", [0.5, 1.0, 2.5])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [100, 5001, 300001])
def test_rows_of_extreme_values(V, dtype, tau):
    z, ids, t, dl = rows(V, 12, dtype, V)
    zd, idd, td = z.cuda(), ids.cuda(), t.cuda()
    loss, lse = fwd(zd, idd, td, tau)
    wl, wm, ws, wd, wdm = reference(z, ids, t, dl, tau)
    # every difference to the row's largest logit is 0, an ordinary one or infinite, so an ordinary row's count holds
    n = roundings(z[4, :V // 2], t[0], tau, V)
    ref64.assert_close(loss, wl, wm, n, "loss")
    # a logit over tau of the type's range rounds to infinity where it leaves float32; two roundings and the result's own
    ws32 = ws.float().double()
    ref64.assert_close(lse, ws32, 1 + ws32.abs().nan_to_num(posinf=0.0), n, "lse")
    dz = torch.full_like(zd, 5.0)
    dg.det_topk_distill_bwd(dz, zd, idd, td, lse, dl.cuda(), tau=tau)
    ref64.assert_close(dz, wd, wdm, n, "dlogits")


def test_ordinary_rows_beside_extreme_ones_keep_their_bits():
    z, ids, t, dl = rows(20000, 12, F32, 1)
    alone = [x[4:5].contiguous().cuda() for x in (z, ids, t)]
    want = fwd(*alone)
    got = fwd(z.cuda(), ids.cuda(), t.cuda())
    assert torch.equal(got[0][4:5], want[0]) and torch.equal(got[1][4:5], want[1])


@pytest.mark.parametrize("shift", [-1e4, -1100.0, 1100.0, 9000.0])
def test_rows_far_from_zero_keep_their_digits(shift):
    """Float32 gradients of rows whose lse has few digits left for log s."""
    g = torch.Generator().manual_seed(2)
    z = torch.randn(3, 9001, generator=g) + shift
    z[2] = shift
    ids = torch.stack([torch.randperm(9001, generator=g)[:9] for _ in range(3)]).int()
    t, dl = torch.randn(3, 9, generator=g) * 3, torch.randn(3, generator=g) + 3
    loss, lse = fwd(z.cuda(), ids.cuda(), t.cuda())
    dz = torch.zeros_like(z).cuda()
    dg.det_topk_distill_bwd(dz, z.cuda(), ids.cuda(), t.cuda(), lse, dl.cuda())
    wl, wm, _, wd, wdm = reference(z, ids, t, dl, 1.0)
    # the differences to the largest logit are those of an ordinary row
    n = roundings(z - shift, t, 1.0, 9001)
    ref64.assert_close(loss, wl, wm, n, "loss")
    ref64.assert_close(dz, wd, wdm, n, "dlogits")
