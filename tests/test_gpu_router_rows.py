"""Sigmoid scores of det_router_balance: a row's results depend on that row alone,
and rows of negative logits keep the scores that are small beside their largest."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64
from tests.test_gpu_router_balance import BF, F32, fwd, make, offsets

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [3, 8, 24, 64, 300])
def test_a_rows_bits_do_not_depend_on_its_neighbours(E, dtype):
    """Every second row replaced by very negative ones: the others keep their gradients' bits."""
    z, _ = make(64, E, 2, dtype, E)
    counts = torch.randint(0, 90, (1, E), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    out = []
    for low in (0.0, 150.0, 45.0):
        x = z.clone()
        x[1::2] -= low
        dz = torch.zeros_like(x).cuda()
        dg.det_router_balance_bwd(dz, x.cuda(), offsets(0, 64), counts.cuda(), torch.ones(1, device="cuda"), 2, score="sigmoid")
        out.append(dz[::2].clone())
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


@pytest.mark.parametrize("E", [2, 16, 40])
def test_small_scores_beside_small_scores(E):
    """Rows whose largest logit is anywhere from -120 to 5 and whose others lie up to 66 below it (a ratio of e^-66 =
    2^-95): p against float64, one row per segment so that prob_sum is the row's p."""
    T = 251
    top = torch.linspace(-120.0, 5.0, T)
    z = top[:, None] - torch.linspace(0.0, 66.0, E)[None]
    offs = torch.arange(T + 1, dtype=torch.int32)
    ids = torch.zeros(T, 1, dtype=torch.int32)
    _, _, psum = fwd(z.cuda(), ids.cuda(), offs.cuda(), score="sigmoid")
    want = ref64.router_probs(z, "sigmoid")
    # the exponents' arguments reach 66 + 120 in either form (a difference, a product), exp's 3, the row's sum and quotient
    ref64.assert_close(psum, want, want, 3 * (66 + 120) + 30, "prob_sum")
    # a count for the smallest score: its gradient p (1 - p) (1 - sigmoid) is of the size of p
    counts = torch.zeros(T, E, dtype=torch.int32)
    counts[:, -1] = 1
    dz = torch.zeros_like(z).cuda()
    dg.det_router_balance_bwd(dz, z.cuda(), offs.cuda(), counts.cuda(), torch.ones(T, device="cuda"), 1, score="sigmoid")
    wd, wm = ref64.router_bwd(z, offs.tolist(), counts, torch.ones(T), 1, 1.0, "sigmoid", torch.zeros(T, E))
    ref64.assert_close(dz, wd, wm, 3 * (66 + 120) + 60, "dlogits")
