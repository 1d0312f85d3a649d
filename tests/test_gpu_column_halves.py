"""Outputs that are column ranges of one buffer, beside each other or beside an input's
range: no element overlaps, so the calls take them and give the bits of separate buffers."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests.test_gpu_block_norm import bwd, dev, fwd, make
from tests.test_gpu_router_balance import offsets

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T,D", [(5, 64), (33, 203), (7, 9000), (1, 8)])
def test_block_norm(T, D, dtype):
    d = dev(make(T, D, dtype, seed=T))
    o = fwd(d)
    want = bwd(d, o)
    # f and gate are the halves of one projection's output, and so are their gradients and y and h
    both = torch.cat([d["f"], d["gate"]], 1)
    e = dict(d, f=both[:, :D], gate=both[:, D:])
    yh, g3 = torch.full((T, 2 * D), 9.0, device="cuda").to(dtype), torch.full((T, 3 * D + 5), 9.0, device="cuda").to(dtype)
    o2 = fwd(e, outs=dict(o, y=yh[:, :D], h=yh[:, D:]))
    assert all(torch.equal(o2[k], o[k]) for k in o)
    dw = {k: torch.zeros(D, device="cuda") for k in ("dw_post", "dalpha", "dw_pre")}
    r = dict(dgate=g3[:, :D], dx=g3[:, D:2 * D], df=g3[:, 2 * D:3 * D])
    dg.det_block_norm_bwd(e["dy"], e["x"], e["f"], r["dx"], r["df"], dh=e["dh"], gate=e["gate"], w_post=e["w_post"],
                          alpha=e["alpha"], w_pre=e["w_pre"], rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"],
                          dgate=r["dgate"], **dw)
    assert all(torch.equal(v, want[k]) for k, v in {**r, **dw}.items())
    assert bool((g3[:, 3 * D:] == 9).all())
    if T > 1:
        # one shared column, whichever comes first, is refused
        for a, b in ((g3[:, :D], g3[:, D - 1:2 * D - 1]), (g3[:, D - 1:2 * D - 1], g3[:, :D])):
            with pytest.raises(dg.DetError, match="overlap"):
                dg.det_block_norm_bwd(e["dy"], e["x"], e["f"], a, b)


def test_router_and_distillation_gradients_beside_their_logits():
    g = torch.Generator().manual_seed(1)
    buf = torch.zeros(30, 130, device="cuda")
    z, dz = buf[:, 3:43], buf[:, 80:120]
    z.copy_(torch.randn(30, 40, generator=g))
    counts, one = torch.randint(0, 9, (1, 40), dtype=torch.int32, generator=g).cuda(), torch.ones(1, device="cuda")
    want = torch.zeros(30, 40, device="cuda")
    dg.det_router_balance_bwd(want, z, offsets(0, 30), counts, one, 2)
    dg.det_router_balance_bwd(dz, z, offsets(0, 30), counts, one, 2)
    assert torch.equal(dz, want)
    ids = torch.randint(0, 40, (30, 4), dtype=torch.int32, generator=g).cuda()
    t, w = torch.randn(30, 4, generator=g).cuda(), torch.ones(30, device="cuda")
    loss, lse = torch.zeros(30, device="cuda"), torch.zeros(30, device="cuda")
    dg.det_topk_distill(z, ids, t, loss, lse)
    dg.det_topk_distill_bwd(want, z, ids, t, lse, w)
    dg.det_topk_distill_bwd(dz, z, ids, t, lse, w)
    assert torch.equal(dz, want)
    with pytest.raises(dg.DetError, match="overlap"):
        dg.det_topk_distill_bwd(buf[:, 42:82], z, ids, t, lse, w)
