"""det_router_balance with several workgroups per segment, whose sums meet in a
workspace from the allocator: captured into graphs, and on two streams at once."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests.test_gpu_router_balance import BF, fwd, make, offsets

pytestmark = pytest.mark.gpu


def test_workspaces_in_graphs_and_on_two_streams():
    T, E, K = 5000, 96, 4
    assert dg.det_router_balance_workspace_size(T, E, K, 3) > 0
    z, ids = (t.cuda() for t in make(T, E, K, BF, 21))
    od = offsets(0, 1000, 1000, 4990)
    counts = torch.zeros(3, E, dtype=torch.int32, device="cuda")
    psum, loss, dz = torch.zeros(3, E, device="cuda"), torch.zeros(3, device="cuda"), torch.zeros_like(z)
    one = torch.ones(3, device="cuda")

    def step():
        dg.det_router_balance(z, ids, od, counts, psum, loss, coeff=0.5)
        dg.det_router_balance_bwd(dz, z, od, counts, one, K, coeff=0.5)
    graphs = []
    for _ in range(2):      # each graph has a workspace of its own
        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for r in range(5):
        z.mul_(0.9)
        step()
        want = [t.clone() for t in (loss, counts, psum, dz)]
        for g in graphs:
            for t in (loss, counts, psum, dz):
                t.fill_(7)
            torch.empty(1 << 22, device="cuda").normal_()    # eager work between the replays
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(dz[4990:], torch.full_like(dz[4990:], 7))
            dz[4990:] = want[3][4990:]
            assert all(torch.equal(a, b) for a, b in zip((loss, counts, psum, dz), want)), r
    # two streams at once, each call with a workspace of its own from the allocator
    want = [t.clone() for t in fwd(z, ids, od, 0.5)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for r in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                bufs = (torch.zeros(3, device="cuda"), torch.zeros_like(counts), torch.zeros_like(psum))
            dg.det_router_balance(z, ids, od, bufs[1], bufs[2], bufs[0], coeff=0.5, stream=s)
            outs.append(bufs)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))
