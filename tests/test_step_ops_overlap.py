"""Rows with strides in one buffer: what shares an element is refused, whichever of the
two comes first and however the strides relate (CPU only, no kernel launches)."""
import os

import pytest

import deterministic_gradient_reductions_amd as dg
from tests.test_step_ops_abi import A, DISTILL_BWD, NORM, NORM_BWD, OVERLAP, P, ROUTER_BWD, run

pytestmark = pytest.mark.skipif(not os.path.exists(dg.library_path), reason="libdetgrad.so not built")


def at(p, elements):
    return P(p.value + 2 * elements)    # bf16


@pytest.mark.parametrize("fn,args", [
    # one shared column: the second's start in the first, the first's start in the second, and over the row's end
    ("det_block_norm_bwd", dict(NORM_BWD, dx_ld=200, df_ld=200, df=at(A[10], 63))),
    ("det_block_norm_bwd", dict(NORM_BWD, dx_ld=200, df_ld=200, dx=at(A[11], 63))),
    ("det_block_norm_bwd", dict(NORM_BWD, dx_ld=200, df_ld=200, df=at(A[10], 137))),
    ("det_block_norm_bwd", dict(NORM_BWD, dx_ld=200, df_ld=200, df=at(A[10], 3 * 200 + 63))),
    # beside each other in one row, with different strides
    ("det_block_norm_bwd", dict(NORM_BWD, dx_ld=200, df_ld=201, df=at(A[10], 64))),
    # a gate per token in another's columns
    ("det_block_norm_bwd", dict(NORM_BWD, gate_cols=1, gate_ld=1, dgate_ld=200, dx_ld=200, dgate=at(A[10], 63))),
    ("det_block_norm", dict(NORM, y_ld=130, h_ld=130, h=at(A[6], 67))),
    ("det_block_norm", dict(NORM, x_ld=130, y_ld=130, y=at(A[0], 3))),
    ("det_router_balance_bwd", dict(ROUTER_BWD, ld=128, ld_d=128, dlogits=at(A[1], 65))),
    ("det_topk_distill_bwd", dict(DISTILL_BWD, ld=60000, ld_d=60000, dlogits=at(A[1], 29999))),
    # a whole vector in a gap between columns is still inside the rows' span
    ("det_block_norm", dict(NORM, y_ld=200, rstd_pre=P(A[6].value + 2 * 64))),
])
def test_shared_elements_are_refused(fn, args):
    assert run(fn, args) == OVERLAP, dg.lib().det_last_error()
