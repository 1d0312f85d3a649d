"""Float64 references of the gated delta rule and of the query and key norms, on the
CPU, written token by token from the formulas.

Magnitudes. An output of the delta rule is a chain of products over a chunk and over
the chunks before it; its rounding errors are sums of many independent ones, each at
most half a step of a float32 value on the path. `delta` and `delta_bwd` give for
every output the size of what such a value can be, by Cauchy-Schwarz from the largest
norms that occur (per call and head): scale |q| |S column| for o, and so on. With n
roundings on the path the error's standard deviation is below sqrt(n) 2^-24 of that;
the tests allow eight of them. The norms count their roundings one by one.
"""
from __future__ import annotations

import math

import numpy as np
import torch

from tests.ref64 import assert_close, bounds

#: Roundings of one chunk on an output's path: sums over 128 channels and three times over 64 tokens, their
#: operands' words.
PER_CHUNK = 128 + 3 * 64 + 16


def allowed(chunks):
    return 8.0 * math.sqrt(PER_CHUNK * (chunks + 1))


def _heads(x, H):
    return x.double().repeat_interleave(H // x.shape[1], dim=1)


def _norms(s):
    """Largest column, row and whole norms of [H, dk, dv], per head."""
    return torch.stack([s.norm(dim=1).amax(1), s.norm(dim=2).amax(1), s.flatten(1).norm(dim=1)])


def delta(q, k, v, g, beta, offs, s0, scale):
    """o [T, H, dv] (NaN in rows of no sequence), s1 [S, H, dk, dv], magnitudes, and what the backward needs."""
    T, H = v.shape[:2]
    q, k, v, g, beta = _heads(q, H), _heads(k, H), v.double(), g.double().clamp(min=-1e4), beta.double()
    b = bounds(offs, T)
    S = len(b) - 1
    o, s1, tape = torch.full(v.shape, math.nan, dtype=torch.float64), [], []
    most = torch.zeros(3, H, dtype=torch.float64)
    for s in range(S):
        st = s0[s].double() if s0 is not None else torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64)
        for t in range(b[s], b[s + 1]):
            kept = st * g[t].exp()[:, None, None]
            n = v[t] - (k[t][:, :, None] * kept).sum(1)
            u = beta[t][:, None] * n
            tape.append((s, t, st, kept, n, u))
            st = kept + k[t][:, :, None] * u[:, None, :]
            o[t] = scale * (q[t][:, :, None] * st).sum(1)
            most = torch.maximum(most, torch.maximum(_norms(st), _norms(k[t][:, :, None] * u[:, None, :])))
        s1.append(st)
    s1 = torch.stack(s1) if s1 else torch.zeros((0, H, q.shape[2], v.shape[2]), dtype=torch.float64)
    qn = abs(scale) * q.norm(dim=2).amax(0) if T else torch.zeros(H).double()
    mags = dict(o=(qn * most[0])[None, :, None].expand_as(o), s1=most[0][None, :, None, None].expand_as(s1))
    return o, s1, mags, dict(tape=tape, most=most, q=q, k=k, v=v, g=g, beta=beta, b=b, scale=scale)


def delta_bwd(do, x, ds1, group):
    """Gradients and magnitudes from `x`, what delta() kept: dict of dq, dk, dv, dg, dbeta, ds0."""
    q, k, v, beta, scale = x["q"], x["k"], x["v"], x["beta"], x["scale"]
    do = do.double()
    T, H = v.shape[:2]
    nan = dict(fill_value=math.nan, dtype=torch.float64)
    r = dict(dq=torch.full(q.shape, **nan), dk=torch.full(k.shape, **nan), dv=torch.full(v.shape, **nan),
             dg=torch.full((T, H), **nan), dbeta=torch.full((T, H), **nan))
    S = len(x["b"]) - 1
    ds0 = [ds1[s].double() if ds1 is not None else torch.zeros(H, q.shape[2], v.shape[2], dtype=torch.float64)
           for s in range(S)]
    most, un, dn, bn = torch.zeros(3, H).double(), torch.zeros(H).double(), torch.zeros(H).double(), torch.zeros(H).double()
    for s, t, st, kept, n, u in reversed(x["tape"]):
        ds = ds0[s]
        after = kept + k[t][:, :, None] * u[:, None, :]
        r["dq"][t] = scale * (after * do[t][:, None, :]).sum(2)
        ds = ds + scale * q[t][:, :, None] * do[t][:, None, :]
        most = torch.maximum(most, _norms(ds))
        du = (k[t][:, :, None] * ds).sum(1)
        r["dv"][t] = beta[t][:, None] * du
        r["dbeta"][t] = (du * n).sum(1)
        r["dk"][t] = (ds * u[:, None, :]).sum(2) - (kept * r["dv"][t][:, None, :]).sum(2)
        ds = ds - k[t][:, :, None] * r["dv"][t][:, None, :]
        r["dg"][t] = (ds * kept).sum((1, 2))
        ds0[s] = ds * x["g"][t].exp()[:, None, None]
        un, dn = torch.maximum(un, u.norm(dim=1)), torch.maximum(dn, r["dv"][t].norm(dim=1))
        bn = torch.maximum(bn, du.norm(dim=1) * n.norm(dim=1))
    r["ds0"] = torch.stack(ds0) if ds0 else torch.zeros((0, H, q.shape[2], v.shape[2]), dtype=torch.float64)
    S_col, S_row, S_all = x["most"]
    one = torch.ones(H).double()
    m = dict(dq=abs(scale) * do.norm(dim=2).amax(0) * S_row if T else one, dk=most[1] * un + S_row * dn + most[0] * un,
             dv=most[0], dg=most[2] * S_all, dbeta=bn + most[0] * un, ds0=most[0])
    mags = {n: (m[n][None, :, None, None] if r[n].dim() == 4 else m[n][None, :, None] if r[n].dim() == 3 else m[n][None])
            .expand_as(r[n]) for n in r}
    for n in ("dq", "dk"):
        r[n] = r[n].unflatten(1, (-1, group)).sum(2)
        mags[n] = mags[n].unflatten(1, (-1, group)).sum(2)
    return r, mags


# ------------------------------------------------------------- dg, token by token
def delta_dg_mag(x, do, s0, ds1):
    """dg's magnitude [T, H] from `x`, what delta() kept: dg of token t is <dS', exp(g) S> of the gradient and the state
    on its two sides, and a chunk forms it as the sum of the products of what either is made of, each with the decays
    between the two, that of t among them. By Cauchy-Schwarz these are at most the product of two sums of norms, of the
    terms of S_{t-1} (the first state, k u^T with |u| <= beta (|v| + |k| |S'|)) and of dS'_t (the last gradient, scale
    q do^T, k dN^T with |dN| <= beta |k| |dS|), each decayed up to its side of t."""
    q, k, v, g, beta, scale = (x[n] for n in ("q", "k", "v", "g", "beta", "scale"))
    T, H = v.shape[:2]
    norm = lambda s: s.flatten(1).norm(dim=1)  # noqa: E731
    zero = torch.zeros(H).double()
    mag, before, sums, grads = torch.zeros(T, H).double(), {}, {}, {}
    for s, t, st, kept, n, u in x["tape"]:
        if s not in sums:
            sums[s] = norm(s0[s].double()) if s0 is not None else zero
        before[t] = g[t].exp() * sums[s]
        un = beta[t] * (v[t].norm(dim=1) + k[t].norm(dim=1) * norm(kept))
        sums[s] = before[t] + k[t].norm(dim=1) * un
    ds = {}
    for s, t, st, kept, n, u in reversed(x["tape"]):
        if s not in ds:
            ds[s] = ds1[s].double() if ds1 is not None else torch.zeros_like(st)
            grads[s] = norm(ds[s])
        d = ds[s] + scale * q[t][:, :, None] * do[t].double()[:, None, :]
        kn = k[t].norm(dim=1)
        after = grads[s] + abs(scale) * q[t].norm(dim=1) * do[t].double().norm(dim=1) + kn * beta[t] * kn * norm(d)
        mag[t] = before[t] * after
        grads[s] = g[t].exp() * after
        d = d - k[t][:, :, None] * (beta[t][:, None] * (k[t][:, :, None] * d).sum(1))[:, None, :]
        ds[s] = d * g[t].exp()[:, None, None]
    return mag


# ------------------------------------------------------------ query and key norms
def turns(pos, inv_freq, axis):
    """cos and sin [T, 1, R / 2], from angles with 64 bits of fraction (the product of 31 and 24 bits, exactly); an axis
    that there is not turns by nothing."""
    pos = pos if pos.dim() == 2 else pos[None]
    axis = torch.zeros(inv_freq.shape, dtype=torch.long) if axis is None else axis.long()
    there = ((axis >= 0) & (axis < pos.shape[0])).numpy()
    assert np.finfo(np.longdouble).nmant >= 63
    a = pos[axis.clamp(0, pos.shape[0] - 1)].numpy().astype(np.longdouble).T * inv_freq.numpy().astype(np.longdouble)
    a = np.where(there, a, np.longdouble(0.0))
    return tuple(torch.from_numpy(f(a).astype(np.float64))[:, None] for f in (np.cos, np.sin))


def turn(x, cs, pairs):
    """x with its first channels turned; with sn negated, turned back."""
    if cs is None:
        return x
    c, s = cs
    R = 2 * c.shape[-1]
    i = torch.arange(R // 2)
    a, b = (i, i + R // 2) if pairs == "halves" else (2 * i, 2 * i + 1)
    y = x.clone()
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def turn_mag(x, cs, pairs):
    """The sum of a turned channel's two terms without their signs."""
    return x.abs() if cs is None else turn(x.abs(), (cs[0].abs(), -cs[1].abs()), pairs).maximum(
        turn(x.abs(), (cs[0].abs(), cs[1].abs()), pairs))


def _rstd(x, norm, eps):
    s = x.square().sum(-1, keepdim=True)
    return torch.ones_like(s) if norm == "none" else 1.0 / torch.sqrt((s / x.shape[-1] if norm == "rms" else s) + eps)


def qk(x, w, norm, eps, cs, pairs):
    """One side's output and magnitude."""
    x = x.double()
    n = x * _rstd(x, norm, eps) * (1.0 if w is None else w.double())
    return turn(n, cs, pairs), turn_mag(n, cs, pairs)


def qk_bwd(dy, x, w, norm, eps, cs, pairs):
    """dx, its magnitude, dw, its magnitude."""
    back = None if cs is None else (cs[0], -cs[1])
    x, dy = x.double(), dy.double()
    d, dm = turn(dy, back, pairs), turn_mag(dy, back, pairs)
    r = _rstd(x, norm, eps)
    xh, w = x * r, torch.ones(x.shape[-1]).double() if w is None else w.double()
    u, um = d * w, dm * w.abs()
    if norm == "none":
        dx, mag = u, um
    else:
        inv = 1.0 / x.shape[-1] if norm == "rms" else 1.0
        dx = r * (u - xh * (u * xh).sum(-1, keepdim=True) * inv)
        mag = r * (um + xh.abs() * (um * xh.abs()).sum(-1, keepdim=True) * inv)
    return dx, mag, (d * xh).sum((0, 1)), (dm * xh.abs()).sum((0, 1))


__all__ = ["allowed", "assert_close", "bounds", "delta", "delta_bwd", "delta_dg_mag", "qk", "qk_bwd", "turn", "turn_mag", "turns"]
