"""Measured cases of the gated delta rule and of the norms of queries and keys with their rotation.

Each case is one pass through one operator: its forward ("fwd"), its forward and
backward in turn ("step"), or, for the delta rule, one new token per sequence
against a cache of states ("token"). With ``own`` false, ``run`` computes the
operator from elementary torch operations; with ``own`` true it makes the
library's calls.

Gated delta rule (T tokens of S packed sequences, Hk key heads, H value heads, per value head a state S [dk, dv]):
    S' = exp(g_t) S_{t-1};  u_t = beta_t (v_t - S'^T k_t);  S_t = S' + k_t u_t^T;  o_t = scale S_t^T q_t
Query and key norms (T tokens, Hq + Hk heads of D channels):
    n = w x / sqrt(mean(x^2) + eps)  ("l2": the sum in place of the mean)
    y = n with the pairs of its first R channels turned by the angles pos * inv_freq, pos one of A axes by pair
"""
from __future__ import annotations

import math

import torch

own = False

DEVICE = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}
EPS = 1e-6
CHUNK = 64          # tokens per chunk of the plain form


# ---------------------------------------------------------------------- cases
def listed():
    return [
        # three sequences of a small model decoding one token each: launch latency
        dict(name="delta_token_small", op="delta", dir="token", dtype="f32", T=3, N=5, Hk=2, H=4, dim_k=64, dim_v=64),
        # a serving batch, two value heads per key head: every state is read and written once
        dict(name="delta_token_serve", op="delta", dir="token", dtype="bf16", T=128, N=160, Hk=16, H=32, dim_k=128, dim_v=128),
        # a few short ragged prompts, head sizes that are no power of two, float32
        dict(name="delta_fwd_odd", op="delta", dir="fwd", dtype="f32", T=333, S=5, Hk=3, H=3, dim_k=48, dim_v=80),
        # one long prompt: the recurrence has nothing to run beside it but the heads and the columns of the state
        dict(name="delta_fwd_long", op="delta", dir="fwd", dtype="bf16", T=32768, S=1, Hk=16, H=32, dim_k=128, dim_v=128),
        # one training microbatch of float32 inputs, odd sizes
        dict(name="delta_step_odd", op="delta", dir="step", dtype="f32", T=2999, S=7, Hk=5, H=5, dim_k=96, dim_v=100),
        # the largest: eight packed sequences, 16 Ki tokens, every gradient
        dict(name="delta_step_train", op="delta", dir="step", dtype="bf16", T=16384, S=8, Hk=16, H=32, dim_k=128, dim_v=128),
        # four tokens of a decoding batch: launch latency
        dict(name="qk_fwd_tokens", op="qk", dir="fwd", dtype="bf16", T=4, Hq=32, Hk=8, D=128, R=128, axes=1,
             pairs="halves", norm="rms", weights=True),
        # a prefill or training microbatch, four queries per key
        dict(name="qk_fwd_train", op="qk", dir="fwd", dtype="bf16", T=16384, Hq=32, Hk=8, D=128, R=128, axes=1,
             pairs="halves", norm="rms", weights=True),
        # images and video: three position axes (time, height, width), an odd number of tokens
        dict(name="qk_step_axes", op="qk", dir="step", dtype="bf16", T=8191, Hq=16, Hk=2, D=128, R=128, axes=3,
             pairs="halves", norm="rms", weights=True),
        # a rotation of half of an uncommon head size, neighbouring pairs, float32
        dict(name="qk_step_odd", op="qk", dir="step", dtype="f32", T=1501, Hq=7, Hk=3, D=80, R=40, axes=1,
             pairs="neighbours", norm="rms", weights=True),
        # the delta rule's own queries and keys: unit length, no rotation, no weights
        dict(name="qk_step_unit", op="qk", dir="step", dtype="bf16", T=32768, Hq=16, Hk=16, D=128, R=0, axes=0,
             pairs="halves", norm="l2", weights=False),
    ]


def _log_int(rng, lo, hi):
    """A whole number in [lo, hi], uniform in its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if rng.random() < 0.5:
        case = dict(op="delta", dir=rng.choice(["token", "fwd", "step"]), dtype=dtype)
        Hk = _log_int(rng, 1, 16)
        H = Hk * rng.choice([1, 1, 2, 3])
        dk, dv = rng.choice([64, 128, rng.randint(16, 128)]), rng.choice([64, 128, rng.randint(16, 128)])
        if case["dir"] == "token":
            T = _log_int(rng, 1, max(1, min(256, 4096 // H)))
            case.update(T=T, N=T + rng.randint(0, 32))
        else:
            T = _log_int(rng, 1, min(16384, 131072 // H))
            case.update(T=T, S=_log_int(rng, 1, min(12, T)))
        case.update(Hk=Hk, H=H, dim_k=dk, dim_v=dv)
        return case
    D = 2 * rng.randint(8, 128) if rng.random() < 0.5 else rng.choice([64, 128, 256])
    Hk = _log_int(rng, 1, 16)
    Hq = Hk * rng.choice([1, 2, 4, 7])
    axes = rng.choice([0, 1, 1, 3])
    R = 0 if axes == 0 else rng.choice([D, D, 2 * rng.randint(1, D // 2)])
    return dict(op="qk", dir=rng.choice(["fwd", "step"]), dtype=dtype, T=_log_int(rng, 1, min(32768, (1 << 25) // (D * (Hq + Hk)))),
                Hq=Hq, Hk=Hk, D=D, R=R, axes=axes, pairs=rng.choice(["halves", "neighbours"]),
                norm=rng.choice(["rms", "rms", "l2", "none"]), weights=rng.random() < 0.8)


# --------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEVICE) * scale).to(dtype)


def _prepare_delta(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, Hk, H, dk, dv = c["T"], c["Hk"], c["H"], c["dim_k"], c["dim_v"]
    st = dict(c)
    # queries and keys of unit length that share a direction per head, as a layer's do
    for name in ("q", "k"):
        x = _normal(g, (T, Hk, dk)) + 0.7 * _normal(g, (1, Hk, dk))
        st[name] = (x / x.square().sum(-1, keepdim=True).sqrt()).to(dt)
    st["v"] = _normal(g, (T, H, dv), dt)
    # decays of a gate: from heads that keep hundreds of tokens to heads that forget in one
    A_log = torch.rand((H,), generator=g, device=DEVICE) * 6.0 - 5.0
    bias = torch.rand((H,), generator=g, device=DEVICE) * 2.0 - 1.0
    st["g"] = -torch.exp(A_log) * torch.log1p(torch.exp(_normal(g, (T, H)) + bias))
    st["beta"] = torch.sigmoid(_normal(g, (T, H), scale=1.5)).to(dt)
    st["scale"] = dk ** -0.5
    st["o"] = torch.zeros((T, H, dv), dtype=dt, device=DEVICE)      # tokens of no sequence keep these zeros
    h = torch.Generator()
    h.manual_seed(seed)
    if c["dir"] == "token":
        st["state"] = _normal(g, (c["N"], H, dk, dv), scale=0.3)
        slots = torch.randperm(c["N"], generator=h)[:T].to(torch.int32)
        if T >= 8:
            slots[int(torch.randint(0, T, (1,), generator=h))] = -1  # a row of a padded batch
        st["slots"] = slots.to(DEVICE)
        return st
    S = c["S"]
    # S ragged sequences (some may be empty), and a few padding tokens at the end
    last = T - int(torch.randint(0, T // 256 + 1, (1,), generator=h))
    even = [last * (i + 1) // S for i in range(S - 1)]
    move = (torch.rand((S - 1,), generator=h) - 0.5) * (last / S)
    cuts = sorted(max(0, min(last, int(e + m))) for e, m in zip(even, move.tolist()))
    st["cuts"] = [0] + cuts + [last]
    st["offs"] = torch.tensor(st["cuts"], dtype=torch.int32, device=DEVICE)
    st["s0"] = _normal(g, (S, H, dk, dv), scale=0.1)
    st["s1"] = torch.zeros_like(st["s0"])
    if c["dir"] == "step":
        st["do"] = _normal(g, (T, H, dv), dt, 0.1)
        st["ds1"] = _normal(g, (S, H, dk, dv), scale=0.01)
        st["ds0"] = torch.zeros_like(st["s0"])
        for name in ("q", "k", "v", "beta"):
            st["d" + name] = torch.zeros_like(st[name])
        st["dg"] = torch.zeros_like(st["beta"])
    return st


def _prepare_qk(c, seed):
    g, dt = _gen(seed), DTYPES[c["dtype"]]
    T, Hq, Hk, D, R, A = c["T"], c["Hq"], c["Hk"], c["D"], c["R"], c["axes"]
    st = dict(c)
    # queries and keys are column ranges of one projection's output, which holds the values too
    qkv = _normal(g, (T, Hq + 2 * Hk, D), dt)
    st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    for name in ("w_q", "w_k"):
        st[name] = 1.0 + _normal(g, (D,), scale=0.1) if c["weights"] else None
    st["pos"] = st["inv_freq"] = st["axis"] = None
    if R:
        st["inv_freq"] = 1e6 ** (-torch.arange(0, R, 2, device=DEVICE, dtype=torch.float64) / R)
        st["inv_freq"] = st["inv_freq"].to(torch.float32)
        start = int(torch.randint(0, 100000, (1,), generator=g, device=DEVICE))
        t = torch.arange(T, device=DEVICE)
        # one axis: a prompt that continues a long context; three: frames of 24 x 32 patches
        pos = torch.stack([t + start]) if A == 1 else torch.stack([start + t // 768, t // 32 % 24, t % 32])
        st["pos"] = pos.to(torch.int32).contiguous()
        if A > 1:
            # time takes the first quarter of the pairs, height and width the rest in halves
            p = torch.arange(R // 2, device=DEVICE) * 8 // (R // 2)
            st["axis"] = torch.where(p < 2, 0, torch.where(p < 5, 1, 2)).to(torch.int32)
    st["yq"], st["yk"] = (torch.zeros((T, h, D), dtype=dt, device=DEVICE) for h in (Hq, Hk))
    if c["dir"] == "step":
        st["dyq"], st["dyk"] = (_normal(g, (T, h, D), dt, 0.1) for h in (Hq, Hk))
        dqkv = torch.zeros_like(qkv)
        st["dq"], st["dk"] = dqkv[:, :Hq], dqkv[:, Hq:Hq + Hk]
    return st


def prepare(case, seed):
    return {"delta": _prepare_delta, "qk": _prepare_qk}[case["op"]](case, seed)


# ---------------------------------------------------- plain forms: delta rule
def _heads(x, H):
    """[..., Hk, d] -> [..., H, d]: each key head for its H / Hk value heads."""
    return x.repeat_interleave(H // x.shape[-2], dim=-2)


def _token_plain(st):
    H, slots = st["H"], st["slots"].long()
    used = (slots >= 0)[:, None, None]
    at = slots.clamp(min=0)
    q, k, v = _heads(st["q"].float(), H), _heads(st["k"].float(), H), st["v"].float()
    s = st["state"][at]
    kept = s * torch.exp(st["g"])[:, :, None, None]
    u = st["beta"].float()[:, :, None] * (v - (kept * k[..., None]).sum(-2))
    new = kept + k[..., None] * u[..., None, :]
    o = st["scale"] * (new * q[..., None]).sum(-2)
    st["o"].copy_(torch.where(used, o, torch.zeros_like(o)))
    live = (slots >= 0).nonzero()[:, 0]
    st["state"][slots[live]] = new[live]
    return st["o"], st["state"]


def _padded(st):
    """Token indices [S, L] of the sequences, padded to whole chunks, and which of them are tokens."""
    n = st["offs"][1:].long() - st["offs"][:-1].long()
    L = -(-max(1, max(b - a for a, b in zip(st["cuts"], st["cuts"][1:]))) // CHUNK) * CHUNK
    j = torch.arange(L, device=DEVICE)
    real = j[None] < n[:, None]
    return torch.where(real, st["offs"][:-1].long()[:, None] + j[None], torch.zeros_like(j)[None]), real


def _chunks(x, at, real):
    """[T, H, d] -> [S, H, L / CHUNK, CHUNK, d] in float32, zeros where no token is."""
    x = torch.where(real[..., None, None], x[at].to(torch.promote_types(x.dtype, torch.float32)), 0)
    return x.unflatten(1, (-1, CHUNK)).permute(0, 3, 1, 2, 4).contiguous()


def _tokens(x, real, out, at):
    """The reverse of _chunks, rounded into `out`, whose other rows stay as they are."""
    x = x.permute(0, 2, 3, 1, 4).flatten(1, 2)
    out[at[real]] = x[real].to(out.dtype)
    return out


def _tr(x):
    return x.transpose(-1, -2)


def _delta_plain(st):
    H = st["H"]
    at, real = _padded(st)
    q, k = (_chunks(_heads(st[n], H), at, real) for n in ("q", "k"))
    v, beta = _chunks(st["v"], at, real), _chunks(st["beta"][..., None], at, real)
    q = q * st["scale"]
    G = _chunks(st["g"][..., None].double(), at, real).cumsum(-2)                 # [S, H, n, C, 1]
    i = torch.arange(CHUNK, device=DEVICE)
    D = torch.exp(torch.where(i[:, None] >= i[None], G - _tr(G), -math.inf)).float()
    eG, eL, rest = torch.exp(G).float(), torch.exp(G[..., -1:, :]).float(), torch.exp(G[..., -1:, :] - G).float()
    strict = (i[:, None] > i[None]).float()
    M = k @ _tr(k) * D * strict
    P = q @ _tr(k) * D
    MB = M * _tr(beta)
    X = torch.eye(CHUNK, device=DEVICE).expand_as(M).clone()                       # (I + M B)^-1, row by row
    for r in range(1, CHUNK):
        X[..., r:r + 1, :r] = -(MB[..., r:r + 1, :r] @ X[..., :r, :r])
    s, first, new = st["s0"], [], []
    for n in range(v.shape[2]):
        first.append(s)
        new.append(X[:, :, n] @ (v[:, :, n] - eG[:, :, n] * (k[:, :, n] @ s)))
        s = eL[:, :, n] * s + _tr(k[:, :, n]) @ (rest[:, :, n] * beta[:, :, n] * new[n])
    s0, N = torch.stack(first, 2), torch.stack(new, 2)
    U = beta * N
    o = _tokens(eG * (q @ s0) + P @ U, real, torch.zeros_like(st["o"]), at)
    if st["dir"] == "fwd":
        return o, s
    do = _chunks(st["do"], at, real)
    ds, last, dnew, dus = st["ds1"], [], [], []
    for n in reversed(range(v.shape[2])):
        last.append(ds)
        dus.append(_tr(P[:, :, n]) @ do[:, :, n] + rest[:, :, n] * (k[:, :, n] @ ds))
        dnew.append(_tr(X[:, :, n]) @ (beta[:, :, n] * dus[-1]))
        ds = eL[:, :, n] * ds + _tr(eG[:, :, n] * q[:, :, n]) @ do[:, :, n] - _tr(eG[:, :, n] * k[:, :, n]) @ dnew[-1]
    ds1, dN, dU = (torch.stack(x[::-1], 2) for x in (last, dnew, dus))
    XN = dN @ _tr(N) * strict
    dP = do @ _tr(U) * (D > 0)
    dM = -XN * _tr(beta)
    qs, ks, kd = eG * (do @ _tr(s0)), eG * (dN @ _tr(s0)), rest * (U @ _tr(ds1))
    dq = qs + dP * D @ k
    dk = kd - ks + _tr(dP * D) @ q + (dM * D + _tr(dM * D)) @ k
    db = (dU * N).sum(-1, keepdim=True) - _tr((M * XN).sum(-2, keepdim=True))
    E = (dP * P + dM * M).double()
    w = (k * kd).sum(-1, keepdim=True, dtype=torch.float64)
    dG = E.sum(-1, keepdim=True) - _tr(E.sum(-2, keepdim=True)) - w
    dG = dG + (q * qs).sum(-1, keepdim=True, dtype=torch.float64) - (k * ks).sum(-1, keepdim=True, dtype=torch.float64)
    dG[..., -1:, :] += w.sum(-2, keepdim=True) + (eL * s0 * ds1).sum((-1, -2), keepdim=True, dtype=torch.float64)
    dg = dG.flip(-2).cumsum(-2).flip(-2)
    group = (st["Hk"], H // st["Hk"])
    out = {n: torch.zeros_like(st[n]) for n in ("dq", "dk", "dv", "dg", "dbeta")}
    _tokens((dq * st["scale"]).unflatten(1, group).sum(2), real, out["dq"], at)
    _tokens(dk.unflatten(1, group).sum(2), real, out["dk"], at)
    _tokens(dN, real, out["dv"], at)
    _tokens(dg, real, out["dg"][..., None], at)
    _tokens(db, real, out["dbeta"][..., None], at)
    return o, s, ds, *out.values()


# ---------------------------------------------- plain forms: norms and rotation
def _turns(st):
    """cos and sin [T, 1, R / 2] of the angles, which far positions need 64 bits for."""
    axis = st["axis"].long() if st["axis"] is not None else torch.zeros_like(st["inv_freq"], dtype=torch.long)
    a = (st["pos"].double()[axis] * st["inv_freq"].double()[:, None]).t()[:, None]
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, st):
    """The two halves of the rotated pairs, and the channels behind them."""
    R = st["R"]
    a, b = (x[..., :R // 2], x[..., R // 2:R]) if st["pairs"] == "halves" else (x[..., 0:R:2], x[..., 1:R:2])
    return a, b, x[..., R:]


def _joined(a, b, rest, st):
    ab = torch.cat([a, b], -1) if st["pairs"] == "halves" else torch.stack([a, b], -1).flatten(-2)
    return torch.cat([ab, rest], -1)


def _rstd(x, st):
    s = x.square().sum(-1, keepdim=True)
    return torch.rsqrt((s / st["D"] if st["norm"] == "rms" else s) + EPS)


def _qk_plain_fwd(st, x, w, turns):
    n = x.float()
    if st["norm"] != "none":
        n = n * _rstd(n, st)
    if w is not None:
        n = n * w
    if turns:
        (a, b, rest), (c, s) = _pairs(n, st), turns
        n = _joined(a * c - b * s, b * c + a * s, rest, st)
    return n.to(x.dtype)


def _qk_plain_bwd(st, dy, x, w, turns):
    d, xh, dw = dy.float(), x.float(), None
    if turns:
        (a, b, rest), (c, s) = _pairs(d, st), turns
        d = _joined(a * c + b * s, b * c - a * s, rest, st)
    r = _rstd(xh, st) if st["norm"] != "none" else 1.0
    xh = xh * r
    if w is not None:
        dw = (d * xh).sum((0, 1), dtype=torch.float64).float()
        d = d * w
    if st["norm"] != "none":
        m = (d * xh).sum(-1, keepdim=True)
        d = r * (d - xh * (m / st["D"] if st["norm"] == "rms" else m))
    return d.to(x.dtype), dw


def _qk_plain(st):
    turns = _turns(st) if st["R"] else None
    out = tuple(_qk_plain_fwd(st, st[n], st["w_" + n], turns) for n in ("q", "k"))
    if st["dir"] == "fwd":
        return out
    (dq, dwq), (dk, dwk) = (_qk_plain_bwd(st, st["dy" + n], st[n], st["w_" + n], turns) for n in ("q", "k"))
    return out + (dq, dk) + ((dwq, dwk) if st["weights"] else ())


# -------------------------------------------------------------- library calls
def _run_own(st):
    import deterministic_gradient_reductions_amd as dg
    if st["op"] == "qk":
        kw = dict(norm=st["norm"], eps=EPS, pos=st["pos"], inv_freq=st["inv_freq"], axis=st["axis"], pairs=st["pairs"])
        dg.det_qk_norm(st["q"], st["k"], st["yq"], st["yk"], w_q=st["w_q"], w_k=st["w_k"], **kw)
        if st["dir"] == "fwd":
            return st["yq"], st["yk"]
        # the parameter gradients accumulate: a step starts them at zero
        dw = torch.zeros((2, st["D"]), device=DEVICE) if st["weights"] else (None, None)
        dg.det_qk_norm_bwd(st["dyq"], st["dyk"], st["q"], st["k"], st["dq"], st["dk"], w_q=st["w_q"], w_k=st["w_k"],
                           dw_q=dw[0], dw_k=dw[1], **kw)
        return (st["yq"], st["yk"], st["dq"], st["dk"]) + ((dw[0], dw[1]) if st["weights"] else ())
    x = (st["q"], st["k"], st["v"], st["g"], st["beta"])
    if st["dir"] == "token":
        dg.det_delta_rule_step(*x, st["state"], st["o"], slots=st["slots"], scale=st["scale"])
        return st["o"], st["state"]
    states = None
    if st["dir"] == "step":
        shape = dg.det_delta_rule_states_shape(st["q"], st["v"], st["offs"])
        states = torch.empty(shape, device=DEVICE)
    dg.det_delta_rule(*x, st["o"], st["offs"], initial_state=st["s0"], final_state=st["s1"], states=states,
                      scale=st["scale"])
    if st["dir"] == "fwd":
        return st["o"], st["s1"]
    dg.det_delta_rule_bwd(st["do"], *x, st["offs"], states, st["dq"], st["dk"], st["dv"], st["dg"], st["dbeta"],
                          dfinal_state=st["ds1"], dinitial_state=st["ds0"], scale=st["scale"])
    return st["o"], st["s1"], st["ds0"], st["dq"], st["dk"], st["dv"], st["dg"], st["dbeta"]


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "qk":
        return _qk_plain(state)
    return _token_plain(state) if state["dir"] == "token" else _delta_plain(state)


# ----------------------------------------------------------------------- work
def work(case):
    c, b, T = case, BYTES[case["dtype"]], case["T"]
    if c["op"] == "qk":
        n = T * (c["Hq"] + c["Hk"]) * c["D"]
        # a step's backward needs the inputs that its forward has read already
        bytes_ = n * b * (2 if c["dir"] == "fwd" else 4) + 4 * T * c["axes"] + 2 * c["R"] + 8 * c["D"] * int(c["weights"])
        return {"bytes": bytes_, "flops": n * (8 if c["dir"] == "fwd" else 24)}
    Hk, H, dk, dv = c["Hk"], c["H"], c["dim_k"], c["dim_v"]
    qk, v, gates, state = 2 * T * Hk * dk * b, T * H * dv * b, T * H, H * dk * dv
    if c["dir"] == "token":
        return {"bytes": qk + 2 * v + gates * (4 + b) + 2 * T * state * 4, "flops": 7 * T * state}
    fwd = qk + 2 * v + gates * (4 + b) + 2 * c["S"] * state * 4
    bwd = qk + 2 * v + gates * 2 * b + 2 * c["S"] * state * 4
    step = c["dir"] == "step"
    return {"bytes": fwd + (bwd if step else 0), "flops": T * state * (7 + (16 if step else 0))}


# -------------------------------------------------------------- 64-bit values
def _exact_token(st):
    r = st["H"] // st["Hk"]
    state, o = st["state"].double(), torch.zeros(st["o"].shape, dtype=torch.float64, device=DEVICE)
    for b, slot in enumerate(st["slots"].tolist()):
        if slot < 0:
            continue
        k, q = (torch.stack([st[n][b, h // r].double() for h in range(st["H"])]) for n in ("k", "q"))
        s = state[slot] * st["g"][b].double().exp()[:, None, None]
        u = (st["v"][b].double() - torch.einsum("hk,hkv->hv", k, s)) * st["beta"][b].double()[:, None]
        state[slot] = s + torch.einsum("hk,hv->hkv", k, u)
        o[b] = torch.einsum("hk,hkv->hv", q, state[slot]) * st["scale"]
    return o, state


def _exact_delta(st):
    """Token by token, all sequences and heads at once; the backward forms the states of 32 tokens again at a time."""
    f64 = dict(dtype=torch.float64, device=DEVICE)
    S, H, Hk, dk, dv, r = st["S"], st["H"], st["Hk"], st["dim_k"], st["dim_v"], st["H"] // st["Hk"]
    lens = [b - a for a, b in zip(st["cuts"], st["cuts"][1:])]
    L, names = max(lens), ("q", "k", "v", "g", "beta") + (("do",) if st["dir"] == "step" else ())
    x = {}
    for n in names:      # [L, S, heads, ...], zeros behind a sequence's end
        x[n] = torch.zeros((L, S) + st[n].shape[1:], **f64)
        for i, (a, m) in enumerate(zip(st["cuts"], lens)):
            x[n][:m, i] = st[n][a:a + m].double()
    x["a"] = x["g"].exp()[..., None, None]

    def inputs(t):
        return (x["q"][t].repeat_interleave(r, 1), x["k"][t].repeat_interleave(r, 1), x["v"][t], x["a"][t],
                x["beta"][t][..., None])

    def forward(s, t):
        q, k, v, a, b = inputs(t)
        s1 = s * a
        n = v - (k[..., None] * s1).sum(-2)
        return s1, n, s1 + k[..., None] * (b * n)[..., None, :]

    o = torch.zeros((L, S, H, dv), **f64)
    s, marks = st["s0"].double(), []
    for t in range(L):
        if t % 32 == 0:
            marks.append(s)
        s = forward(s, t)[2]
        o[t] = st["scale"] * (x["q"][t].repeat_interleave(r, 1)[..., None] * s).sum(-2)

    def packed(y):
        z = torch.zeros((st["T"],) + y.shape[2:], **f64)
        for i, (a, m) in enumerate(zip(st["cuts"], lens)):
            z[a:a + m] = y[:m, i]
        return z

    if st["dir"] == "fwd":
        return packed(o), s
    dq, dk_, dv_ = (torch.zeros((L, S, H, d), **f64) for d in (dk, dk, dv))
    dg, db = (torch.zeros((L, S, H), **f64) for _ in range(2))
    ds = st["ds1"].double()
    for block in reversed(range(len(marks))):
        kept, c = [], marks[block]
        for t in range(32 * block, min(L, 32 * block + 32)):
            s1, n, c = forward(c, t)
            kept.append((t, s1, n, c))
        for t, s1, n, s_t in reversed(kept):
            q, k, _, a, b = inputs(t)
            do = x["do"][t] * st["scale"]
            dq[t] = (s_t * do[..., None, :]).sum(-1)
            ds = ds + q[..., None] * do[..., None, :]
            du = (k[..., None] * ds).sum(-2)
            dk_[t] = (ds * (b * n)[..., None, :]).sum(-1)
            db[t] = (du * n).sum(-1)
            dv_[t] = b * du
            dk_[t] -= (s1 * dv_[t][..., None, :]).sum(-1)
            ds = ds - k[..., None] * dv_[t][..., None, :]
            dg[t] = (ds * s1).sum((-1, -2))
            ds = ds * a
    shared = [packed(y).unflatten(1, (Hk, r)).sum(2) for y in (dq, dk_)]
    return packed(o), s, ds, *shared, packed(dv_), packed(dg), packed(db)


def _exact_qk(st):
    R, D = st["R"], st["D"]
    if R:
        axis = [0] * (R // 2) if st["axis"] is None else st["axis"].tolist()
        ang = torch.stack([st["pos"][a].double() * st["inv_freq"][i].double() for i, a in enumerate(axis)], 1)[:, None]
        turn = torch.polar(torch.ones_like(ang), ang)
        i = torch.arange(R // 2, device=DEVICE)
        first, second = (i, i + R // 2) if st["pairs"] == "halves" else (2 * i, 2 * i + 1)

    def rotate(x, way):
        if not R:
            return x
        z = torch.complex(x[..., first], x[..., second]) * (turn if way > 0 else turn.conj())
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out, back, dws = [], [], []
    for n in ("q", "k"):
        x = st[n].double()
        w = torch.ones(D, dtype=torch.float64, device=DEVICE) if st["w_" + n] is None else st["w_" + n].double()
        size = {"rms": D, "l2": 1, "none": 1}[st["norm"]]
        rms = 1.0 if st["norm"] == "none" else ((x * x).sum(-1, keepdim=True) / size + EPS) ** 0.5
        out.append(rotate(x / rms * w, 1))
        if st["dir"] == "step":
            d = rotate(st["dy" + n].double(), -1)
            dws.append((d * x / rms).sum((0, 1)))
            dx = d * w / rms
            if st["norm"] != "none":
                dx = dx - x * (d * w * x).sum(-1, keepdim=True) / (size * rms ** 3)
            back.append(dx)
    return (*out, *back, *(dws if st["weights"] else ()))


def exact(case, seed):
    st = prepare(case, seed)
    if st["op"] == "qk":
        return _exact_qk(st)
    return _exact_token(st) if st["dir"] == "token" else _exact_delta(st)
