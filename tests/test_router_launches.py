"""The router's one-launch form is for calls whose single workgroups have little to do:
sizes of its workspace (0 in that form) over tokens, experts, slots and segments."""
import os

import pytest

import deterministic_gradient_reductions_amd as dg

pytestmark = pytest.mark.skipif(not os.path.exists(dg.library_path), reason="libdetgrad.so not built")


@pytest.mark.parametrize("T,E,K,S,one", [
    (48, 8, 2, 3, True), (0, 8, 2, 1, True), (1, 1, 1, 1, True), (4096, 8, 2, 1, True), (256, 256, 8, 1, True),
    (16384, 8, 2, 8, True), (2048, 64, 6, 8, True),
    # few experts, many tokens
    (65536, 2, 2, 1, False), (131072, 1, 1, 1, False), (16384, 8, 2, 1, False), (65536, 2, 2, 64, False),
    # few tokens, many slots
    (16384, 8, 8, 1, False), (1, 2, 65536, 1, False), (200, 4, 3000, 1, False), (200, 4, 3000, 64, False),
    # many columns
    (512, 256, 8, 1, False), (128, 1024, 8, 1, False)])
def test_one_launch_only_where_each_workgroup_has_little_to_do(T, E, K, S, one):
    assert (dg.det_router_balance_workspace_size(T, E, K, S) == 0) == one
