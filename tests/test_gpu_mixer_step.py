"""A token mixer's training step as it is used: unit-length queries and keys (det_qk_norm),
the gated delta rule with the gate's decays, and back to the gate's parameters, whose
column sums are det_colsum's; against float64 autograd of the whole, in a graph too."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg
from tests import ref64_delta as R

pytestmark = pytest.mark.gpu

T, OFFS, Hk, H, DK, DV = 200, [0, 77, 200], 2, 4, 32, 48


def make():
    gen = torch.Generator().manual_seed(3)
    n = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    return dict(q=n(T, Hk, DK), k=n(T, Hk, DK), v=n(T, H, DV), a=n(T, H), b=n(T, H), A_log=torch.rand(H, generator=gen) - 1.5,
                dt_bias=torch.rand(H, generator=gen), w_q=1 + 0.1 * n(DK), w_k=1 + 0.1 * n(DK), do=n(T, H, DV))


def kernels(d, o):
    offs = o["offs"]
    dg.det_qk_norm(d["q"], d["k"], o["qn"], o["kn"], w_q=d["w_q"], w_k=d["w_k"], norm="l2")
    g = -torch.exp(d["A_log"]) * torch.nn.functional.softplus(d["a"] + d["dt_bias"])
    beta = torch.sigmoid(d["b"])
    x = (o["qn"], o["kn"], d["v"], g, beta)
    dg.det_delta_rule(*x, o["o"], offs, states=o["states"])
    dg.det_delta_rule_bwd(d["do"], *x, offs, o["states"], o["dqn"], o["dkn"], o["dv"], o["dg"], o["dbeta"])
    for n in ("dA_log", "ddt_bias", "dw_q", "dw_k"):
        o[n].zero_()
    dg.det_colsum_da(d["a"], o["dg"], d["A_log"], d["dt_bias"], o["dA_log"], o["ddt_bias"], o["da"], ws=o["ws"])
    dg.det_qk_norm_bwd(o["dqn"], o["dkn"], d["q"], d["k"], o["dq"], o["dk"], w_q=d["w_q"], w_k=d["w_k"], dw_q=o["dw_q"],
                       dw_k=o["dw_k"], norm="l2")


def buffers(d):
    z = torch.zeros_like
    o = {n: z(d[m]) for n, m in (("qn", "q"), ("kn", "k"), ("dqn", "q"), ("dkn", "k"), ("dq", "q"), ("dk", "k"), ("o", "v"),
                                 ("dv", "v"), ("dg", "a"), ("dbeta", "a"), ("da", "a"), ("dA_log", "A_log"),
                                 ("ddt_bias", "dt_bias"), ("dw_q", "w_q"), ("dw_k", "w_k"))}
    o["offs"] = torch.tensor(OFFS, dtype=torch.int32).cuda()
    o["states"] = torch.zeros(dg.det_delta_rule_states_shape(d["q"], d["v"], o["offs"]), device="cuda")
    o["ws"] = dg.Workspace(dg.det_colsum_workspace_size(T, H))
    return o


def autograd(h):
    x = {n: t.double().requires_grad_(n != "do") for n, t in h.items()}
    unit = lambda t, w: t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() * w  # noqa: E731
    q, k = (unit(x[n], x["w_" + n]).repeat_interleave(H // Hk, 1) for n in "qk")
    g = -torch.exp(x["A_log"]) * torch.nn.functional.softplus(x["a"] + x["dt_bias"])
    beta, rows = torch.sigmoid(x["b"]), []
    beta.retain_grad()
    for s0, s1 in zip(OFFS, OFFS[1:]):
        S = torch.zeros(H, DK, DV, dtype=torch.float64)
        for t in range(s0, s1):
            S = S * g[t].exp()[:, None, None]
            u = beta[t][:, None] * (x["v"][t] - (k[t][:, :, None] * S).sum(1))
            S = S + k[t][:, :, None] * u[:, None, :]
            rows.append(DK ** -0.5 * (q[t][:, :, None] * S).sum(1))
    o = torch.stack(rows)
    (o * x["do"]).sum().backward()
    return o.detach(), {n: t.grad for n, t in x.items() if n != "do"}, beta.grad


def test_step_against_float64_and_in_a_graph():
    h = make()
    d = {n: t.cuda() for n, t in h.items()}
    o = buffers(d)
    kernels(d, o)
    want, grads, dbeta = autograd(h)

    def near(got, ref, what):
        # 2^-24 times the roundings' share in the sums of the chain (R.allowed), relative to the largest value
        tol = 2.0 ** -24 * 4 * R.allowed(4) * float(ref.abs().max())
        err = float((got.cpu().double() - ref).abs().max())
        assert err <= tol, (what, err, tol)
    near(o["o"], want, "o")
    near(o["dbeta"], dbeta, "dbeta")
    for n, m in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("da", "a"), ("dA_log", "A_log"), ("ddt_bias", "dt_bias"),
                 ("dw_q", "w_q"), ("dw_k", "w_k")):
        near(o[n], grads[m], n)
    first = {n: t.clone() for n, t in o.items() if torch.is_tensor(t)}
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kernels(d, o)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        kernels(d, o)
    other = buffers(d)
    for i in range(4):
        for n in ("o", "dq", "dk", "dv", "dw_q", "dA_log", "da"):
            o[n].fill_(float(i))
        g.replay()
        kernels(d, other)
        torch.cuda.synchronize()
        for n, t in first.items():
            assert torch.equal(o[n], t) and torch.equal(other[n], t), n
