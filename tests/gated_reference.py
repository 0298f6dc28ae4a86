"""Plain float64 form of the gated recurrence and its gradients, token by token
(numpy), with a bound on each output's fp32 error.

The bounds.  One fp32 step h = a h + b has a relative error of at most u = 2^-24
in the fma, and a and w carry the gate's: the gate's argument g + bias is one
rounding of a number below 16 in size (at most 16 u absolute, once in the
product with log2 e and once in the exponential's own error), which moves a by
a (1 - a) and w by at most w times it; exp2, rcp, sqrt and the products add a
handful of u.  A token's error lives tau = 1 / (1 - a) tokens, so a state is
off by at most (2 tau + 64) u times hbar, the same recurrence run on |w x|; the
adjoint likewise, and a product of the two by the sum.  The tests draw gates
with tau <= 100: K = 600 covers a product of both, 300 one of them.
"""
import numpy as np

U = 2.0 ** -24
K1, K2 = 300 * U, 600 * U


def sigmoid(v):
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1 / (1 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1 + np.exp(-np.abs(v))))


def gates(gate, gate_bias, rate, mode):
    """a, w, da/dv, da/drate, dw/da, shaped as gate; parameters (dim,)."""
    bias = 0.0 if gate_bias is None else np.asarray(gate_bias, np.float64)[:, None]
    v = np.asarray(gate, np.float64) + bias
    s, t = sigmoid(v), sigmoid(-v)
    if rate is None:
        a, om, da, dr = s, t, s * t, None
    else:
        c = np.asarray(rate, np.float64)[:, None]
        a, om = np.exp(-c * s), -np.expm1(-c * s)
        da, dr = -c * a * s * t, -a * s
    if mode == "plain":
        w, dw = np.ones_like(a), np.zeros_like(a)
    elif mode == "convex":
        w, dw = om, -np.ones_like(a)
    else:
        w = np.sqrt(om * (1 + a))
        with np.errstate(divide="ignore", invalid="ignore"):
            dw = np.where(w > 0, -a / w, 0.0)
    return a, w, da, dr, dw


def forward(x, gate, gate_bias=None, rate=None, z=None, reset=None, h0=None, mode="plain"):
    """dict: y, last, states, and the bounds y_err, last_err (fp32 arithmetic only)."""
    x = np.asarray(x, np.float64)
    a, w, _, _, _ = gates(gate, gate_bias, rate, mode)
    batch, dim, L = x.shape
    drop = np.zeros((batch, 1, L), bool) if reset is None else np.asarray(reset).astype(bool)[:, None, :]
    drop = drop | (a == 0)
    h = np.zeros((batch, dim)) if h0 is None else np.asarray(h0, np.float64)
    bar = np.abs(h)
    states, bars = np.empty_like(x), np.empty_like(x)
    with np.errstate(invalid="ignore", over="ignore"):
        for t in range(L):
            b = w[..., t] * x[..., t]
            h = np.where(drop[..., t], b, a[..., t] * h + b)
            bar = np.where(drop[..., t], np.abs(b), a[..., t] * bar + np.abs(b))
            states[..., t], bars[..., t] = h, bar
        sz = 1.0 if z is None else np.asarray(z, np.float64) * sigmoid(np.asarray(z, np.float64))
        return dict(y=states * sz, last=states[..., -1].copy(), states=states, bars=bars,
                    y_err=K1 * bars * np.abs(sz), last_err=K1 * bars[..., -1])


def backward(x, gate, dy, gate_bias=None, rate=None, z=None, reset=None, h0=None, dlast=None, mode="plain"):
    """dict of gradients and, under name + "_err", their bounds."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    f = forward(x, gate, gate_bias, rate, z, reset, h0, mode)
    a, w, da, dr, dw = gates(gate, gate_bias, rate, mode)
    batch, dim, L = x.shape
    drop = np.zeros((batch, 1, L), bool) if reset is None else np.asarray(reset).astype(bool)[:, None, :]
    drop = np.broadcast_to(drop, x.shape) | (a == 0)
    out = {}
    q = dy
    if z is not None:
        zz = np.asarray(z, np.float64)
        sg = sigmoid(zz)
        ds = sg * (1 + zz * (1 - sg))
        out["dz"] = dy * f["states"] * ds
        out["dz_err"] = K1 * np.abs(dy) * f["bars"] * (np.abs(ds) + sg)
        q = dy * zz * sg
    carry = np.zeros((batch, dim)) if dlast is None else np.asarray(dlast, np.float64)
    lam, lbar = np.empty_like(x), np.empty_like(x)
    cbar = np.abs(carry)
    for t in range(L - 1, -1, -1):
        lam[..., t], lbar[..., t] = q[..., t] + carry, np.abs(q[..., t]) + cbar
        carry = np.where(drop[..., t], 0.0, a[..., t] * lam[..., t])
        cbar = np.where(drop[..., t], 0.0, a[..., t] * lbar[..., t])
    out["dh0"], out["dh0_err"] = carry, K1 * cbar
    out["dx"], out["dx_err"] = lam * w, K1 * lbar * w
    start = np.zeros((batch, dim)) if h0 is None else np.asarray(h0, np.float64)
    hp = np.concatenate([start[..., None], f["states"][..., :-1]], -1)
    hb = np.concatenate([np.abs(start)[..., None], f["bars"][..., :-1]], -1)
    hp, hb = np.where(drop, 0.0, hp), np.where(drop, 0.0, hb)
    la = lam * (hp + x * dw)
    labar = lbar * (hb + np.abs(x * dw))
    out["dgate"], out["dgate_err"] = la * da, K2 * labar * np.abs(da)
    # sums over batch and tokens: the terms' own errors, and the additions' (a tree of at most 64 levels of u)
    out["dgate_bias"] = out["dgate"].sum((0, 2))
    out["dgate_bias_err"] = (out["dgate_err"] + 64 * U * np.abs(out["dgate"])).sum((0, 2))
    if rate is not None:
        out["drate"] = (la * dr).sum((0, 2))
        out["drate_err"] = ((K2 + 64 * U) * labar * np.abs(dr)).sum((0, 2))
    return out
