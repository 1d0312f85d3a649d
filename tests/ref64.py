"""Float64 references of the router balance loss, the top-logit distillation
and the block norms, on the CPU, written from the formulas.

Each reference returns values and, for the tolerances, magnitudes: the same
expression with every term replaced by its absolute value. A float32 evaluation
with n roundings on the path of a value differs from it by at most about
n * 2^-24 * magnitude; the result's own rounding adds half a step of its type.
"""
from __future__ import annotations

import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TINY = 2.0 ** -126   # results below the smallest normal float32 may lose digits


def assert_close(got, want, mag, roundings, what):
    """|got - want| <= roundings * 2^-24 * mag + half a step of got's type * |want| + TINY, NaN and inf alike."""
    g, w = got.detach().cpu().double(), want.double()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    special = ~torch.isfinite(w)
    same = (g == w) | (torch.isnan(g) & torch.isnan(w))
    assert bool(same[special].all()), "%s: NaN or infinity differs" % what
    tol = roundings * U * mag.double() + HALF_STEP[got.dtype] * w.abs() + TINY
    err = (g - w).abs()
    bad = (~special) & ~(err <= tol)
    if bool(bad.any()):
        i = int(torch.where(bad, err / tol, torch.zeros_like(err)).nan_to_num(nan=math.inf).argmax())
        raise AssertionError("%s: %d of %d outside; worst at %d: got %r want %r, tolerance %.3g" % (
            what, int(bad.sum()), g.numel(), i, g.flatten()[i].item(), w.flatten()[i].item(),
            tol.flatten()[i].item()))


# --------------------------------------------------------------- router balance
def bounds(offs, T):
    b = []
    for o in offs:
        b.append(max(min(max(int(o), 0), T), b[-1] if b else 0))
    return b


def router_probs(z, score):
    """p [T, E]; a row of -inf only has p = 0."""
    l = z.double()
    if score == "sigmoid":
        l = torch.nn.functional.logsigmoid(l)
    empty = (l == -math.inf).all(1, keepdim=True)
    return torch.where(empty, torch.zeros_like(l), torch.softmax(l, 1))


def router(z, ids, offs, coeff, score):
    """(loss, counts, prob_sum) with p's magnitudes being p itself (all terms are positive)."""
    T, E = z.shape
    K = ids.shape[1]
    p = router_probs(z, score)
    b = bounds(offs, T)
    S = len(b) - 1
    loss, counts, psum = torch.zeros(S).double(), torch.zeros(S, E, dtype=torch.int32), torch.zeros(S, E).double()
    for s in range(S):
        n = b[s + 1] - b[s]
        if n == 0:
            continue
        for e in range(E):
            counts[s, e] = int((ids[b[s]:b[s + 1]] == e).sum())
        psum[s] = p[b[s]:b[s + 1]].sum(0)
        loss[s] = coeff * E / (K * float(n) ** 2) * (counts[s].double() * psum[s]).sum()
    return loss, counts, psum


def router_bwd(z, offs, counts, dloss, K, coeff, score, old):
    """(dlogits, magnitude); rows of no segment keep `old`."""
    T, E = z.shape
    p = router_probs(z, score)
    b = bounds(offs, T)
    out, mag = old.double().clone(), torch.zeros(T, E).double()
    for s in range(len(b) - 1):
        n = b[s + 1] - b[s]
        if n == 0:
            continue
        rows = slice(b[s], b[s + 1])
        c = counts[s].double()
        g = float(dloss[s]) * coeff * E / (K * float(n) ** 2)
        q = p[rows]
        d = g * q * (c - (q * c).sum(1, keepdim=True))
        # the kernel subtracts the whole mean count K n / E from every count first
        r = (c - K * n // E).abs()
        m = abs(g) * q * (r + (q * r).sum(1, keepdim=True))
        if score == "sigmoid":
            f = torch.sigmoid(-z[rows].double())
            d, m = d * f, m * f
        out[rows], mag[rows] = d, m
    return out, mag


# ----------------------------------------------------------------- distillation
def teacher(ids, t, V, tau):
    """q [T, K] and log q, over the valid slots; zeros in a row without teacher mass."""
    ok = (ids >= 0) & (ids < V)
    x = torch.where(ok, t.double() / tau, torch.full(t.shape, -math.inf).double())
    live = (x > -math.inf).any(1, keepdim=True) | (ok & t.isnan()).any(1, keepdim=True)
    x = torch.where(live, x, torch.zeros_like(x))
    lq = torch.log_softmax(x, 1) if x.shape[1] else x
    q = torch.where(live & ok, lq.exp(), torch.zeros_like(lq))
    return q, torch.where(q == 0, torch.zeros_like(lq), lq)


def distill(z, ids, t, tau):
    """(loss, its magnitude, lse)."""
    T, V = z.shape
    x = z.double() / tau
    lse = torch.logsumexp(x, 1)
    q, lq = teacher(ids, t, V, tau)
    safe = ids.clamp(0, V - 1).long()
    xk = x.gather(1, safe)
    zero = torch.zeros_like(q)
    loss = torch.where(q == 0, zero, q * (lq - xk + lse[:, None])).sum(1)
    mag = torch.where(q == 0, zero, q * (lq.abs() + xk.abs() + lse.abs()[:, None])).sum(1)
    return loss, mag, lse


def distill_bwd(z, ids, t, lse, dloss, tau):
    """(dlogits, magnitude)."""
    T, V = z.shape
    q, _ = teacher(ids, t, V, tau)
    live = (q.sum(1, keepdim=True) != 0) & (dloss.double() != 0)[:, None]
    p = torch.exp(z.double() / tau - lse.double()[:, None])
    y = torch.zeros(T, V).double().scatter_add(1, ids.clamp(0, V - 1).long(), q)
    a = (dloss.double() / tau)[:, None]
    zero = torch.zeros_like(p)
    return torch.where(live, a * (p - y), zero), torch.where(live, a.abs() * (p + y), zero)


# ------------------------------------------------------------------ block norms
def norm(x, f, gate, w_post, alpha, w_pre, eps):
    """dict of values and "_mag" magnitudes: y, h, rstd_post, rstd_pre."""
    x, f = x.double(), f.double()
    one = torch.ones(x.shape[1]).double()
    al = one if alpha is None else alpha.double()
    s = torch.ones(x.shape[0], 1).double() if gate is None else torch.sigmoid(gate.double())
    out = {}
    n = f
    if w_post is not None:
        out["rstd_post"] = rp = (f.square().mean(1) + eps).rsqrt()
        n = f * rp[:, None] * w_post.double()
    b = al * s * n
    out["y"], out["y_mag"] = x + b, x.abs() + b.abs()
    if w_pre is not None:
        out["rstd_pre"] = rq = (out["y"].square().mean(1) + eps).rsqrt()
        out["h"] = out["y"] * rq[:, None] * w_pre.double()
        out["h_mag"] = out["y_mag"] * rq[:, None] * w_pre.double().abs()
        # the mean's terms carry y's error: |dy| / rms relative to 1 (mean of |y| y_mag against mean of y^2)
        out["pre_mag"] = (out["y"].abs() * out["y_mag"]).mean(1) * rq ** 2
    return out


def norm_bwd(dy, dh, x, f, gate, w_post, alpha, w_pre, rstd_post, rstd_pre):
    """dict of gradients and "_mag" magnitudes, with the given rstd factors."""
    T, D = f.shape
    f = f.double()
    one = torch.ones(D).double()
    al = one if alpha is None else alpha.double()
    wp = one if w_post is None else w_post.double()
    s = torch.ones(T, 1).double() if gate is None else torch.sigmoid(gate.double())
    rp = torch.ones(T, 1).double() if rstd_post is None else rstd_post.double()[:, None]
    fh = f * rp
    n = fh * wp
    d, dm = dy.double(), dy.double().abs()
    out = {}
    if w_pre is not None:
        rq = rstd_pre.double()[:, None]
        yh = (x.double() + al * s * n) * rq
        ym = (x.double().abs() + (al * s * n).abs()) * rq
        u = w_pre.double() * dh.double()
        d = d + rq * (u - yh * (u * yh).mean(1, keepdim=True))
        dm = dm + rq * (u.abs() + ym * (u.abs() * ym).mean(1, keepdim=True))
        out["dw_pre"], out["dw_pre_mag"] = (dh.double() * yh).sum(0), (dh.double().abs() * ym).sum(0)
    out["dx"], out["dx_mag"] = d, dm
    if alpha is not None:
        out["dalpha"], out["dalpha_mag"] = (d * s * n).sum(0), (dm * s * n.abs()).sum(0)
    dn, dnm = d * al * s, dm * al.abs() * s
    if gate is not None:
        g, gm = dn * n * (1 - s), dnm * n.abs()      # 1 - s: an error of s counts against 1
        if gate.shape[1] == 1 and D > 1:
            g, gm = g.sum(1, keepdim=True), gm.sum(1, keepdim=True)
        out["dgate"], out["dgate_mag"] = g, gm
    v, vm = dn * wp, dnm * wp.abs()
    if w_post is not None:
        out["dw_post"], out["dw_post_mag"] = (dn * fh).sum(0), (dnm * fh.abs()).sum(0)
        v, vm = (rp * (v - fh * (v * fh).mean(1, keepdim=True)),
                 rp * (vm + fh.abs() * (vm * fh.abs()).mean(1, keepdim=True)))
    out["df"], out["df_mag"] = v, vm
    return out
