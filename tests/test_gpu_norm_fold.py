"""The parameter gradients of det_block_norm_bwd: the workgroups' sums are added in
float64, so a large one does not swallow the small ones behind it."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [5, 130, 2048])
@pytest.mark.parametrize("at", [0, 17, 511])
def test_one_large_row_among_512(D, at):
    """dalpha = sum_t dy f: 512 rows (one per workgroup) of 1, one of them 2^24. The sum 2^24 + 511 in float32 is
    2^24 + 512, to the bit; float32 additions behind the large row would lose each 1."""
    f = torch.ones(512, D, device="cuda")
    f[at] = 2.0 ** 24
    dy = torch.ones_like(f)
    dx, df, dalpha = torch.zeros_like(f), torch.zeros_like(f), torch.zeros(D, device="cuda")
    dg.det_block_norm_bwd(dy, None, f, dx, df, alpha=torch.ones(D, device="cuda"), dalpha=dalpha)
    assert bool((dalpha == 2.0 ** 24 + 512).all()), dalpha[:4]
    assert torch.equal(df, dy) and torch.equal(dx, dy)
