"""Measured cases of the router balance loss, the top-logit distillation loss and the block norms.

Each case is one pass through one operator: its forward ("fwd"), its backward
("bwd") or both in turn ("step"). With ``own`` false, ``run`` computes the
operator from elementary torch operations; with ``own`` true it makes the
library's calls.

Router balance (T tokens, E experts, top-K ids, S sequences given by offsets):
    p = softmax(z) or normalised sigmoid(z);  counts[s, e], P[s, e] = sums over the tokens of s
    loss[s] = coeff * E / (K * N_s^2) * sum_e counts[s, e] * P[s, e]
Distillation (T tokens, V words, K teacher slots):
    q = softmax(teacher / tau) over the valid slots, x = student / tau
    loss = sum_k q_k * (log q_k - x[id_k] + logsumexp(x))
Block norm (T tokens, D channels), the boundary between two residual blocks:
    y = x + alpha * sigmoid(gate) * (w_post * f / rms(f));  h = w_pre * y / rms(y)
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # a handful of tokens of three short sequences, eight experts: launch latency
        dict(name="router_step_small", op="router", dir="step", dtype="f32", T=48, E=8, K=2, S=3, score="softmax"),
        # one microbatch of eight sequences, 64 experts
        dict(name="router_fwd_train", op="router", dir="fwd", dtype="bf16", T=16384, E=64, K=6, S=8, score="softmax"),
        # many short ragged sequences, an expert count that is no power of two, float32 logits
        dict(name="router_bwd_ragged", op="router", dir="bwd", dtype="f32", T=9001, E=160, K=6, S=37, score="softmax"),
        # the largest: a packed batch of 64 Ki tokens over 256 experts with sigmoid scores
        dict(name="router_step_large", op="router", dir="step", dtype="bf16", T=65536, E=256, K=8, S=16,
             score="sigmoid"),
        # three tokens against a long vocabulary: the work has to be split along the row
        dict(name="distill_fwd_few", op="distill", dir="fwd", dtype="f32", T=3, V=131072, K=64, tau=1.0),
        # one training microbatch with a 32 Ki vocabulary
        dict(name="distill_step_train", op="distill", dir="step", dtype="bf16", T=4096, V=32768, K=32, tau=2.0),
        # an odd vocabulary: every second row starts off a 4-byte border
        dict(name="distill_bwd_odd", op="distill", dir="bwd", dtype="bf16", T=1021, V=50001, K=100, tau=1.5),
        # the largest: 2^30 logits
        dict(name="distill_step_large", op="distill", dir="step", dtype="bf16", T=8192, V=131072, K=64, tau=1.0),
        # four tokens of a decoding batch: launch latency
        dict(name="norm_fwd_tokens", op="norm", dir="fwd", dtype="bf16", T=4, D=4096, gate="full", post=True, pre=True,
             alpha=True),
        # one training microbatch, a gate per channel
        dict(name="norm_fwd_train", op="norm", dir="fwd", dtype="bf16", T=8192, D=4096, gate="full", post=True,
             pre=True, alpha=True),
        # odd sizes, one gate per token, float32
        dict(name="norm_step_odd", op="norm", dir="step", dtype="f32", T=3001, D=1407, gate="row", post=True, pre=True,
             alpha=True),
        # the largest: wide rows, every gradient
        dict(name="norm_bwd_large", op="norm", dir="bwd", dtype="bf16", T=16384, D=8192, gate="full", post=True,
             pre=True, alpha=True),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["router", "distill", "norm"])
    case = dict(op=op, dir=rng.choice(["fwd", "bwd", "step"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
    if op == "router":
        E = _log_int(rng, 2, 512)
        case.update(T=_log_int(rng, 1, min(65536, (1 << 23) // E)), E=E, K=rng.randint(1, min(8, E)),
                    S=_log_int(rng, 1, 64), score=rng.choice(["softmax", "sigmoid"]))
    elif op == "distill":
        V = _log_int(rng, 1000, 131072)
        case.update(T=_log_int(rng, 1, min(8192, (1 << 29) // V)), V=V, K=_log_int(rng, 1, 256),
                    tau=rng.choice([1.0, 1.5, 2.0, 4.0]))
    else:
        D = _log_int(rng, 32, 8192)
        case.update(T=_log_int(rng, 1, min(16384, (1 << 25) // D)), D=D, gate=rng.choice(["none", "row", "full", "full"]),
                    post=rng.random() < 0.8, pre=rng.random() < 0.8, alpha=rng.random() < 0.7)
    return case


# --------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype, scale=1.0):
    x = torch.randn(shape, generator=g, device="cuda", dtype=dtype)
    return x if scale == 1.0 else x.mul_(scale)


def _prepare_router(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, E, K, S = c["T"], c["E"], c["K"], c["S"]
    st = dict(c)
    # experts of unequal popularity; the router picks each token's K largest logits
    st["logits"] = (_normal(g, (T, E), torch.float32) + 0.5 * _normal(g, (1, E), torch.float32)).to(dt)
    ids = st["logits"].float().topk(K, dim=1).indices.to(torch.int32)
    dropped = torch.rand((T, K), generator=g, device="cuda") < 0.02   # slots over capacity
    st["ids"] = torch.where(dropped, torch.full_like(ids, -1), ids).contiguous()
    # S ragged sequences, some possibly empty, and a few padding tokens at the end
    h = torch.Generator()
    h.manual_seed(seed)
    last = T - int(torch.randint(0, T // 64 + 1, (1,), generator=h))
    cuts = torch.randint(0, last + 1, (S - 1,), generator=h).sort().values.tolist()
    st["cuts"] = [0] + cuts + [last]
    st["offs"] = torch.tensor(st["cuts"], dtype=torch.int32, device="cuda")
    st["coeff"] = 0.01
    st["dloss"] = torch.rand((S,), generator=g, device="cuda") + 0.5
    # the backward alone is given the counts its forward returned
    seg = torch.bucketize(torch.arange(T, device="cuda"), st["offs"][1:].contiguous(), right=True)
    seg = torch.where(torch.arange(T, device="cuda") < last, seg, torch.full_like(seg, S))
    flat = torch.where(st["ids"] >= 0, seg[:, None] * E + st["ids"], torch.full_like(seg, (S + 1) * E)[:, None])
    st["counts"] = torch.bincount(flat.flatten(), minlength=(S + 1) * E + 1)[:S * E].view(S, E).to(torch.int32)
    st["counts_out"] = torch.zeros((S, E), dtype=torch.int32, device="cuda")
    st["prob_sum"] = torch.zeros((S, E), device="cuda")
    st["loss"] = torch.zeros((S,), device="cuda")
    st["dlogits"] = torch.zeros((T, E), dtype=dt, device="cuda")      # padding tokens keep these zeros
    return st


def _prepare_distill(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, V, K = c["T"], c["V"], c["K"]
    st = dict(c)
    st["logits"] = _normal(g, (T, V), dt, 2.0)
    # distinct words per token: one from each of K equal strides of the vocabulary
    step = V // K
    ids = (torch.arange(K, device="cuda") * step)[None] + torch.randint(0, step, (T, K), generator=g, device="cuda")
    # teacher logits falling from slot to slot; the student partly agrees
    t = 12.0 - 4.0 * torch.rand((T, K), generator=g, device="cuda").cumsum(1) / max(1.0, K ** 0.5)
    st["logits"].scatter_add_(1, ids, (0.7 * t).to(dt))
    ids = ids.to(torch.int32)
    ids = torch.where(torch.rand((T, K), generator=g, device="cuda") < 0.02, torch.full_like(ids, -1), ids)
    pad = torch.rand((T, 1), generator=g, device="cuda") < 0.02       # padding tokens
    st["ids"] = torch.where(pad, torch.full_like(ids, -1), ids).contiguous()
    st["teacher"] = t
    st["dloss"] = torch.where(pad[:, 0], torch.zeros(T, device="cuda"), torch.full((T,), c["tau"] ** 2 / T, device="cuda"))
    st["loss"] = torch.zeros((T,), device="cuda")
    st["lse"] = torch.zeros((T,), device="cuda")
    if c["dir"] != "fwd":
        st["dlogits"] = torch.zeros((T, V), dtype=dt, device="cuda")
    if c["dir"] == "bwd":
        for r in range(0, T, 256):
            st["lse"][r:r + 256] = torch.logsumexp(st["logits"][r:r + 256].double() / c["tau"], 1).float()
    return st


def _prepare_norm(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, D = c["T"], c["D"]
    st = dict(c)
    for name in ("x", "f"):
        st[name] = _normal(g, (T, D), dt)
    st["g"] = None if c["gate"] == "none" else _normal(g, (T, D if c["gate"] == "full" else 1), dt)
    for name, used in (("w_post", c["post"]), ("alpha", c["alpha"]), ("w_pre", c["pre"])):
        w = _normal(g, (D,), torch.float32, 0.1)
        st[name] = (w + (0.5 if name == "alpha" else 1.0)) if used else None
    st["dy"] = _normal(g, (T, D), dt, 0.1)
    st["dh"] = _normal(g, (T, D), dt, 0.1) if c["pre"] else None
    z = torch.zeros_like
    st["y"], st["h"] = z(st["x"]), z(st["x"]) if c["pre"] else None
    st["rstd_post"] = torch.zeros((T,), device="cuda") if c["post"] else None
    st["rstd_pre"] = torch.zeros((T,), device="cuda") if c["pre"] else None
    st["dx"], st["df"] = z(st["x"]), z(st["x"])
    st["dg"] = None if st["g"] is None else z(st["g"])
    if c["dir"] == "bwd":
        y, _, rp, rq = _norm_plain_fwd(st)
        for name, r in (("rstd_post", rp), ("rstd_pre", rq)):
            if r is not None:
                st[name].copy_(r[:, 0])
    return st


def prepare(case, seed):
    return {"router": _prepare_router, "distill": _prepare_distill, "norm": _prepare_norm}[case["op"]](case, seed)


# ---------------------------------------------------------------- plain forms
def _segments(st):
    """Each token's sequence (S for none) and the tokens of every sequence, from the device offsets."""
    t = torch.arange(st["T"], device="cuda")
    offs = st["offs"].long()
    inside = (t[:, None] >= offs[None, :-1]) & (t[:, None] < offs[None, 1:])      # [T, S]
    return inside, (offs[1:] - offs[:-1]).double()


def _router_probs(st):
    z = st["logits"].float()
    if st["score"] == "sigmoid":
        z = z.clamp(max=0.0) - torch.log1p(torch.exp(-z.abs()))
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _router_scale(st, n):
    return torch.where(n > 0, st["coeff"] * st["E"] / (st["K"] * n.clamp(min=1.0) ** 2), torch.zeros_like(n))


def _router_plain_fwd(st):
    S, E = st["S"], st["E"]
    inside, n = _segments(st)
    p = _router_probs(st)
    psum = torch.stack([p[a:b].sum(0, dtype=torch.float64) for a, b in zip(st["cuts"], st["cuts"][1:])])
    # tokens of no sequence and dropped slots are counted in one place behind the last expert
    seg = torch.where(inside.any(1), inside.int().argmax(1), torch.full((st["T"],), S, device="cuda"))[:, None]
    slot = torch.where((st["ids"] >= 0) & (seg < S), seg * E + st["ids"], torch.full_like(seg, S * E))
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device="cuda")
    counts.index_add_(0, slot.flatten(), torch.ones_like(slot.flatten(), dtype=torch.int32))
    counts = counts[:S * E].view(S, E)
    loss = _router_scale(st, n) * (counts.double() * psum).sum(1)
    return loss.float(), counts, psum.float()


def _router_plain_bwd(st, counts):
    inside, n = _segments(st)
    p = _router_probs(st)
    c = inside.float() @ counts.float()                                            # [T, E]
    scale = inside.float() @ (_router_scale(st, n) * st["dloss"].double()).float()[:, None]
    d = scale * p * (c - (p * c).sum(1, keepdim=True))
    if st["score"] == "sigmoid":
        d = d / (1.0 + torch.exp(st["logits"].float()))
    return torch.where(inside.any(1, keepdim=True), d, torch.zeros_like(d)).to(st["logits"].dtype)


def _teacher(st):
    valid = (st["ids"] >= 0) & (st["ids"] < st["V"])
    t = torch.where(valid, st["teacher"] / st["tau"], torch.full_like(st["teacher"], -math.inf))
    m = t.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = torch.exp(t - m)
    s = e.sum(1, keepdim=True)
    q = torch.where(s > 0, e / s, torch.zeros_like(e))
    logq = torch.where(q > 0, t - m - torch.log(s), torch.zeros_like(t))
    return valid, q, logq


def _distill_plain_fwd(st):
    x = st["logits"].float() / st["tau"]
    m = x.amax(1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(1, keepdim=True))
    valid, q, logq = _teacher(st)
    xk = x.gather(1, torch.where(valid, st["ids"], torch.zeros_like(st["ids"])).long())
    terms = torch.where(q > 0, q * (logq - xk + lse), torch.zeros_like(q))
    return terms.sum(1), lse[:, 0]


def _distill_plain_bwd(st, lse):
    valid, q, _ = _teacher(st)
    mass = q.sum(1, keepdim=True)
    p = torch.exp(st["logits"].float() / st["tau"] - lse[:, None]) * mass
    p.scatter_add_(1, torch.where(valid, st["ids"], torch.zeros_like(st["ids"])).long(), -q)
    d = p * (st["dloss"] / st["tau"])[:, None]
    return torch.where((st["dloss"] == 0)[:, None], torch.zeros_like(d), d).to(st["logits"].dtype)


def _norm_plain_fwd(st):
    n, rp, rq, h = st["f"].float(), None, None, None
    if st["post"]:
        rp = torch.rsqrt((n * n).mean(1, keepdim=True) + EPS)
        n = n * rp * st["w_post"]
    if st["alpha"] is not None:
        n = n * st["alpha"]
    if st["g"] is not None:
        n = n / (1.0 + torch.exp(-st["g"].float()))
    y = st["x"].float() + n
    if st["pre"]:
        rq = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        h = y * rq * st["w_pre"]
    return y, h, rp, rq


def _norm_plain_bwd(st, rp, rq):
    f = st["f"].float()
    fh = f * rp[:, None] if st["post"] else f
    n = fh * st["w_post"] if st["post"] else fh
    s = 1.0 / (1.0 + torch.exp(-st["g"].float())) if st["g"] is not None else torch.ones((), device="cuda")
    a = st["alpha"] if st["alpha"] is not None else torch.ones((), device="cuda")
    d, dw_pre, dalpha, dg, dw_post = st["dy"].float(), None, None, None, None
    if st["pre"]:
        yh = (st["x"].float() + a * s * n) * rq[:, None]
        dh = st["dh"].float()
        u = dh * st["w_pre"]
        d = d + rq[:, None] * (u - yh * (u * yh).mean(1, keepdim=True))
        dw_pre = (dh * yh).sum(0, dtype=torch.float64).float()
    if st["alpha"] is not None:
        dalpha = (d * s * n).sum(0, dtype=torch.float64).float()
    dn = d * a * s
    if st["g"] is not None:
        dg = dn * n * (1.0 - s)
        dg = (dg.sum(1, keepdim=True) if st["gate"] == "row" else dg).to(st["x"].dtype)
    df = dn
    if st["post"]:
        dw_post = (dn * fh).sum(0, dtype=torch.float64).float()
        u = dn * st["w_post"]
        df = rp[:, None] * (u - fh * (u * fh).mean(1, keepdim=True))
    return d.to(st["x"].dtype), df.to(st["x"].dtype), dg, dw_post, dalpha, dw_pre


def _present(*outs):
    return tuple(o for o in outs if o is not None)


def _run_plain(st):
    d = st["dir"]
    if st["op"] == "router":
        out = _router_plain_fwd(st) if d != "bwd" else ()
        return out if d == "fwd" else out + (_router_plain_bwd(st, out[1] if out else st["counts"]),)
    if st["op"] == "distill":
        out = _distill_plain_fwd(st) if d != "bwd" else ()
        return out if d == "fwd" else out + (_distill_plain_bwd(st, out[1] if out else st["lse"]),)
    out, rp, rq = (), st["rstd_post"], st["rstd_pre"]
    if d != "bwd":
        y, h, rp, rq = _norm_plain_fwd(st)
        rp, rq = (None if r is None else r[:, 0] for r in (rp, rq))
        out = _present(y.to(st["x"].dtype), None if h is None else h.to(st["x"].dtype), rp, rq)
    return out if d == "fwd" else out + _present(*_norm_plain_bwd(st, rp, rq))


# -------------------------------------------------------------- library calls
def _run_own(st):
    import deterministic_gradient_reductions_amd as dg
    d, out = st["dir"], ()
    if st["op"] == "router":
        counts = st["counts"]
        if d != "bwd":
            counts = st["counts_out"]
            dg.det_router_balance(st["logits"], st["ids"], st["offs"], counts, st["prob_sum"], st["loss"],
                                  coeff=st["coeff"], score=st["score"])
            out = (st["loss"], counts, st["prob_sum"])
        if d != "fwd":
            dg.det_router_balance_bwd(st["dlogits"], st["logits"], st["offs"], counts, st["dloss"], st["K"],
                                      coeff=st["coeff"], score=st["score"])
            out += (st["dlogits"],)
        return out
    if st["op"] == "distill":
        if d != "bwd":
            dg.det_topk_distill(st["logits"], st["ids"], st["teacher"], st["loss"], st["lse"], tau=st["tau"])
            out = (st["loss"], st["lse"])
        if d != "fwd":
            dg.det_topk_distill_bwd(st["dlogits"], st["logits"], st["ids"], st["teacher"], st["lse"], st["dloss"],
                                    tau=st["tau"])
            out += (st["dlogits"],)
        return out
    if d != "bwd":
        dg.det_block_norm(st["x"], st["f"], st["y"], gate=st["g"], w_post=st["w_post"], alpha=st["alpha"],
                          w_pre=st["w_pre"], h=st["h"], rstd_post=st["rstd_post"], rstd_pre=st["rstd_pre"], eps=EPS)
        out = _present(st["y"], st["h"], st["rstd_post"], st["rstd_pre"])
    if d != "fwd":
        # the parameter gradients accumulate: a step starts them at zero
        dw = torch.zeros((3, st["D"]), device="cuda")
        dw_post, dalpha, dw_pre = (dw[i] if st[n] is not None else None
                                   for i, n in enumerate(("w_post", "alpha", "w_pre")))
        dg.det_block_norm_bwd(st["dy"], st["x"], st["f"], st["dx"], st["df"], dh=st["dh"], gate=st["g"],
                              w_post=st["w_post"], alpha=st["alpha"], w_pre=st["w_pre"], rstd_post=st["rstd_post"],
                              rstd_pre=st["rstd_pre"], dgate=st["dg"], dw_post=dw_post, dalpha=dalpha, dw_pre=dw_pre)
        out += _present(st["dx"], st["df"], st["dg"], dw_post, dalpha, dw_pre)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------- work
def work(case):
    c, b, d = case, BYTES[case["dtype"]], case["dir"]
    fwd, bwd = d != "bwd", d != "fwd"
    if c["op"] == "router":
        n, se = c["T"] * c["E"], c["S"] * c["E"]
        # a step reads the logits once: the forward's sums need them all before the backward, but nothing else
        bytes_ = n * b + (c["T"] * c["K"] * 4 + se * 8 if fwd else se * 4) + (n * b if bwd else 0) + 8 * c["S"]
        return {"bytes": bytes_, "flops": n * ((6 if fwd else 0) + (10 if bwd else 0))}
    if c["op"] == "distill":
        n, k = c["T"] * c["V"], c["T"] * c["K"]
        bytes_ = n * b + k * 8 + c["T"] * (8 if fwd else 4) + ((n * b + c["T"] * 4) if bwd else 0)
        return {"bytes": bytes_, "flops": n * ((4 if fwd else 0) + (4 if bwd else 0))}
    n = c["T"] * c["D"]
    g = {"none": 0, "row": c["T"], "full": n}[c["gate"]]
    pre, post, par = int(c["pre"]), int(c["post"]), int(c["pre"]) + int(c["post"]) + int(c["alpha"])
    read = 2 * n + g + ((1 + pre) * n if bwd else 0)
    write = ((1 + pre) * n if fwd else 0) + ((2 * n + g) if bwd else 0)
    bytes_ = (read + write) * b + 4 * c["D"] * par * (2 if bwd else 1) + 4 * c["T"] * (pre + post)
    return {"bytes": bytes_, "flops": n * ((12 if fwd else 0) + (30 if bwd else 0))}


# -------------------------------------------------------------- 64-bit values
def _exact_router(st):
    T, E, K = st["T"], st["E"], st["K"]
    z = st["logits"].double()
    score = z.sigmoid() if st["score"] == "sigmoid" else (z - z.max(dim=1, keepdim=True).values).exp()
    p = score / score.sum(dim=1, keepdim=True)
    offs = st["cuts"]
    loss, counts, psum, dz = [], [], [], torch.zeros_like(z)
    for s in range(st["S"]):
        a, b = offs[s], offs[s + 1]
        ids = st["ids"][a:b].flatten().long()
        c = torch.bincount(ids[ids >= 0], minlength=E)
        if st["dir"] == "bwd":
            c = st["counts"][s].long()
        P = p[a:b].sum(dim=0)
        scale = st["coeff"] * E / (K * (b - a) ** 2) if b > a else 0.0
        counts.append(c.to(torch.int32))
        psum.append(P)
        loss.append(scale * torch.dot(c.double(), P))
        cc = c.double()[None]
        if b > a:
            grad = p[a:b] * (cc - p[a:b] @ c.double()[:, None])
            if st["score"] == "sigmoid":
                grad = grad * (1.0 - score[a:b])
            dz[a:b] = grad * (scale * st["dloss"][s].double())
    out = (torch.stack(loss), torch.stack(counts), torch.stack(psum)) if st["dir"] != "bwd" else ()
    return out if st["dir"] == "fwd" else out + (dz,)


def _exact_distill(st):
    T, V, tau = st["T"], st["V"], float(st["tau"])
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    lse = torch.zeros_like(loss)
    dz = torch.empty((T, V), dtype=torch.float64, device="cuda") if st["dir"] != "fwd" else None
    for r in range(0, T, 512):
        rows = slice(r, min(T, r + 512))
        x = st["logits"][rows].double() / tau
        lp = torch.log_softmax(x, dim=1)
        lse[rows] = torch.logsumexp(x, dim=1)
        ids = st["ids"][rows].long()
        ok = ids >= 0
        t = (st["teacher"][rows].double() / tau).masked_fill(~ok, -math.inf)
        live = ok.any(dim=1, keepdim=True)
        q = torch.softmax(t.masked_fill(~live, 0.0), dim=1) * ok
        pos = q > 0
        term = q * (torch.log(q.masked_fill(~pos, 1.0)) - lp.gather(1, ids.clamp(min=0)))
        loss[rows] = term.masked_fill(~pos, 0.0).sum(dim=1)
        if dz is not None:
            y = torch.zeros_like(x).scatter_add(1, ids.clamp(min=0), q)
            scale = (st["dloss"][rows].double() / tau)[:, None]
            dz[rows] = scale * (lp.exp() * live - y)
    out = (loss, lse) if st["dir"] != "bwd" else ()
    return out if st["dir"] == "fwd" else out + (dz,)


def _exact_norm(st):
    T, D = st["T"], st["D"]
    f64 = dict(dtype=torch.float64, device="cuda")
    one = torch.ones(D, **f64)
    wp, al, wq = (one if st[n] is None else st[n].double() for n in ("w_post", "alpha", "w_pre"))
    keep = {n: [] for n in ("y", "h", "rp", "rq", "dx", "df", "dg")}
    dwp, dal, dwq = (torch.zeros(D, **f64) for _ in range(3))
    for r in range(0, T, 1024):
        rows = slice(r, min(T, r + 1024))
        x, f = st["x"][rows].double(), st["f"][rows].double()
        gate = torch.ones((x.shape[0], 1), **f64) if st["g"] is None else torch.sigmoid(st["g"][rows].double())
        rp = 1.0 / torch.sqrt(f.square().mean(dim=1, keepdim=True) + EPS) if st["post"] else None
        fh = f * rp if st["post"] else f
        y = x + al * gate * wp * fh
        rq = 1.0 / torch.sqrt(y.square().mean(dim=1, keepdim=True) + EPS) if st["pre"] else None
        keep["y"].append(y)
        if st["pre"]:
            keep["h"].append(wq * (y * rq))
            keep["rq"].append(rq[:, 0])
        if st["post"]:
            keep["rp"].append(rp[:, 0])
        if st["dir"] == "fwd":
            continue
        d = st["dy"][rows].double()
        if st["pre"]:
            dh, yh = st["dh"][rows].double(), y * rq
            dwq += (dh * yh).sum(dim=0)
            v = wq * dh
            d = d + rq * v - rq * yh * ((v * yh).sum(dim=1, keepdim=True) / D)
        keep["dx"].append(d)
        dal += (d * gate * wp * fh).sum(dim=0)
        dwp += (d * gate * al * fh).sum(dim=0)
        if st["g"] is not None:
            dgate = d * al * wp * fh
            if st["gate"] == "row":
                dgate = dgate.sum(dim=1, keepdim=True)
            keep["dg"].append(dgate * gate * (1.0 - gate))
        v = d * gate * al * wp
        if st["post"]:
            v = rp * v - rp * fh * ((v * fh).sum(dim=1, keepdim=True) / D)
        keep["df"].append(v)
    k = {n: torch.cat(v) if v else None for n, v in keep.items()}
    out = _present(k["y"], k["h"], k["rp"], k["rq"]) if st["dir"] != "bwd" else ()
    if st["dir"] == "fwd":
        return out
    return out + _present(k["dx"], k["df"], k["dg"], dwp if st["post"] else None,
                          dal if st["alpha"] is not None else None, dwq if st["pre"] else None)


def exact(case, seed):
    st = prepare(case, seed)
    return {"router": _exact_router, "distill": _exact_distill, "norm": _exact_norm}[case["op"]](st)
