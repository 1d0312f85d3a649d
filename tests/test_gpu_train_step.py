"""The operators together as a training step uses them: a block boundary's norms
and gate, the router's balance loss, a teacher's top logits put in canonical
order and distilled, and all gradients back to the block's inputs and
parameters, against float64 autograd of the whole step."""
import pytest
import torch

import deterministic_gradient_reductions_amd as dg

pytestmark = pytest.mark.gpu

T, D, E, V, K, KT, EPS, COEFF, TAU = 96, 72, 12, 501, 2, 16, 1e-6, 0.5, 2.0
OFFS = [0, 30, 30, 90]     # three sequences, one empty, and six padding tokens


def inputs():
    g = torch.Generator().manual_seed(0)

    def n(*s):
        return torch.randn(*s, generator=g)
    ids = torch.stack([torch.randperm(V, generator=g)[:KT] for _ in range(T)]).int()
    ids[torch.rand(T, KT, generator=g) < 0.1] = -1
    return dict(x=n(T, D), f=n(T, D), gate=n(T, 1), w_post=1 + 0.1 * n(D), alpha=0.5 + 0.1 * n(D), w_pre=1 + 0.1 * n(D),
                w_router=0.3 * n(D, E), w_words=0.3 * n(D, V), ids=ids, teacher=3 * n(T, KT))


def token_weights():
    w = torch.zeros(T)
    w[OFFS[0]:OFFS[-1]] = TAU ** 2 / (OFFS[-1] - OFFS[0])     # the padding tokens weigh nothing
    return w


class Step:
    """One step with the library's calls; the products between them in float64, rounded to float32."""

    def __init__(self, d):
        self.d = {k: v.cuda() for k, v in d.items()}
        z = torch.zeros
        c = dict(device="cuda")
        self.offs = torch.tensor(OFFS, dtype=torch.int32, **c)
        self.S = len(OFFS) - 1
        self.weights = token_weights().cuda()
        self.ones = torch.ones(self.S, **c)
        self.y, self.h, self.dx, self.df = (z(T, D, **c) for _ in range(4))
        self.rp, self.rq, self.loss, self.lse = (z(T, **c) for _ in range(4))
        self.dgate, self.dw = z(T, 1, **c), z(3, D, **c)
        self.counts = z(self.S, E, dtype=torch.int32, **c)
        self.psum, self.bal = z(self.S, E, **c), z(self.S, **c)
        self.cid, self.ct, self.cp = z(T, KT, dtype=torch.int32, **c), z(T, KT, **c), z(T, KT, **c)
        self.dr, self.dv = z(T, E, **c), z(T, V, **c)

    def run(self):
        d = self.d
        dg.det_block_norm(d["x"], d["f"], self.y, gate=d["gate"], w_post=d["w_post"], alpha=d["alpha"],
                          w_pre=d["w_pre"], h=self.h, rstd_post=self.rp, rstd_pre=self.rq, eps=EPS)
        h = self.h.double()
        r, v = (h @ d["w_router"].double()).float(), (h @ d["w_words"].double()).float()
        top = r.topk(K, dim=1).indices.int()
        dg.det_router_balance(r, top, self.offs, self.counts, self.psum, self.bal, coeff=COEFF)
        dg.det_topk_canonicalize(d["ids"], d["teacher"], self.cid, self.ct, self.cp)
        dg.det_topk_distill(v, self.cid, self.ct, self.loss, self.lse, tau=TAU)
        dg.det_topk_distill_bwd(self.dv, v, self.cid, self.ct, self.lse, self.weights, tau=TAU)
        dg.det_router_balance_bwd(self.dr, r, self.offs, self.counts, self.ones, K, coeff=COEFF)
        dh = (self.dr.double() @ d["w_router"].double().t() + self.dv.double() @ d["w_words"].double().t()).float()
        self.dw.zero_()
        dg.det_block_norm_bwd(torch.zeros_like(dh), d["x"], d["f"], self.dx, self.df, dh=dh, gate=d["gate"],
                              w_post=d["w_post"], alpha=d["alpha"], w_pre=d["w_pre"], rstd_post=self.rp,
                              rstd_pre=self.rq, dgate=self.dgate, dw_post=self.dw[0], dalpha=self.dw[1],
                              dw_pre=self.dw[2])

    def outs(self):
        return dict(loss=self.loss, bal=self.bal, x=self.dx, f=self.df, gate=self.dgate, w_post=self.dw[0],
                    alpha=self.dw[1], w_pre=self.dw[2])


def reference(d):
    """Losses and gradients of the step by float64 autograd on the CPU."""
    p = {k: d[k].double().requires_grad_() for k in ("x", "f", "gate", "w_post", "alpha", "w_pre")}
    n = p["f"] * (p["f"].square().mean(1, keepdim=True) + EPS).rsqrt() * p["w_post"]
    y = p["x"] + p["alpha"] * torch.sigmoid(p["gate"]) * n
    h = y * (y.square().mean(1, keepdim=True) + EPS).rsqrt() * p["w_pre"]
    r, v = h @ d["w_router"].double(), h @ d["w_words"].double()
    top = r.topk(K, dim=1).indices
    prob = torch.softmax(r, 1)
    bal = []
    for a, b in zip(OFFS, OFFS[1:]):
        counts = torch.bincount(top[a:b].flatten(), minlength=E).double()
        bal.append(COEFF * E / (K * max(b - a, 1) ** 2) * (counts * prob[a:b].sum(0)).sum())
    lp = torch.log_softmax(v / TAU, 1)
    ok = d["ids"] >= 0
    t = (d["teacher"].double() / TAU).masked_fill(~ok, float("-inf"))
    q = torch.softmax(t, 1)
    lq = torch.log(q.masked_fill(~ok, 1.0))
    loss = (q * (lq - lp.gather(1, d["ids"].clamp(min=0).long()))).masked_fill(~ok, 0.0).sum(1)
    ((loss * token_weights().double()).sum() + torch.stack(bal).sum()).backward()
    return dict(loss=loss.detach(), bal=torch.stack(bal).detach(), **{k: t.grad for k, t in p.items()})


def test_step_against_float64_autograd():
    """Relative 2-norm per tensor. Each operator's outputs carry at most about 64 roundings (4e-6); a gradient passes
    through six of them (norm, product, loss, loss's gradient, product, norm's gradient): 2.5e-5."""
    d = inputs()
    s = Step(d)
    s.run()
    want = reference(d)
    for k, got in s.outs().items():
        g, w = got.cpu().double(), want[k]
        if k == "loss":        # the padding tokens' losses are computed, and weigh nothing
            g, w = g[:OFFS[-1]], w[:OFFS[-1]]
        err = float((g - w).norm() / w.norm())
        assert err < 2.5e-5, (k, err)
    assert bool((s.dv[OFFS[-1]:] == 0).all()) and bool((s.dr[OFFS[-1]:] == 0).all())


def test_step_bits_do_not_depend_on_the_teachers_slot_order_or_the_run():
    d = inputs()
    s = Step(d)
    s.run()
    want = {k: v.clone() for k, v in s.outs().items()}
    for r in range(3):
        perm = torch.stack([torch.randperm(KT, generator=torch.Generator().manual_seed(100 * r + t)) for t in range(T)])
        e = dict(d, ids=d["ids"].gather(1, perm), teacher=d["teacher"].gather(1, perm))
        o = Step(e)
        o.run()
        # padding slots (ids of -1) come last, in slot order, and are not read: every output is the same
        assert all(torch.equal(v, want[k]) for k, v in o.outs().items()), r


def test_step_in_a_graph():
    d = inputs()
    s = Step(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.run()
    e = Step(d)
    for r in range(4):
        for t in (s, e):
            t.d["f"].mul_(1.1)
        e.run()
        torch.empty(1 << 20, device="cuda").normal_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(v, e.outs()[k]) for k, v in s.outs().items()), r
