"""Plain float64 form of linear attention with a decay for each head and its
gradients (torch on the CPU), token by token, with a bound on each output's error.

Every output is a sum over pairs of tokens (s, t), s <= t, of decay x products;
`size` runs the same recurrences on magnitudes.  A sum of n terms in fp32 is off
by at most n u times the sum of magnitudes, u = 2^-24, in whatever order, and
a rounding made on a partial sum at one token shrinks with the later decays as the
sum does.  A path holds at most seqlen + dk + dv additions, and as many roundings again
of factors (a decay's exponent, up to 150 before the decay is 0, is off by u
of itself, the exponential by 4 u): n = 2 (seqlen + dk + dv) + 160.  In bf16 the
scores and the state are rounded once more for the next product: 2^-8 of their
magnitudes (2^-7 together where both count).
"""
import torch

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def _decays(rate, step, reset, shape):
    step = torch.ones(shape, dtype=torch.float64) if step is None else step.double()
    a = torch.exp(-step * rate.double())
    if reset is not None:
        a = torch.where(reset[..., None] != 0, torch.zeros_like(a), a)
    return step, a


def _carry(a, s):
    """a s, 0 where a is 0 whatever s is."""
    a = a[..., None, None]
    return torch.where(a == 0, torch.zeros_like(s), a * s)


def _shared(x, heads):
    return x.double().repeat_interleave(heads // x.shape[2], 2)


def forward(q, k, v, rate, step=None, reset=None, h0=None, scale=1.0):
    """(y, last_state, states behind every token)."""
    batch, seqlen, heads, dv = v.shape
    q, k, v = _shared(q, heads), _shared(k, heads), v.double()
    _, a = _decays(rate, step, reset, v.shape[:3])
    s = torch.zeros((batch, heads, q.shape[3], dv), dtype=torch.float64) if h0 is None else h0.double()
    y, states = torch.empty_like(v), []
    for t in range(seqlen):
        s = _carry(a[:, t], s) + k[:, t, :, :, None] * v[:, t, :, None, :]
        states.append(s)
        y[:, t] = scale * (q[:, t, :, :, None] * s).sum(2)
    return y, s, states


def backward(q, k, v, rate, dy, step=None, reset=None, h0=None, dlast=None, scale=1.0, states=None):
    batch, seqlen, heads, dv = v.shape
    groups, dk = q.shape[2:]
    if states is None:
        states = forward(q, k, v, rate, step, reset, h0, scale)[2]
    q, k, v, dy = _shared(q, heads), _shared(k, heads), v.double(), dy.double()
    step, a = _decays(rate, step, reset, v.shape[:3])
    first = torch.zeros_like(states[0]) if h0 is None else h0.double()
    r = torch.zeros_like(first) if dlast is None else dlast.double()
    dq, dkk, dvv, dg = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v), torch.empty_like(a)
    for t in range(seqlen - 1, -1, -1):
        before = states[t - 1] if t else first
        r = r + scale * q[:, t, :, :, None] * dy[:, t, :, None, :]
        dq[:, t] = scale * (states[t] * dy[:, t, :, None, :]).sum(3)
        dkk[:, t] = (r * v[:, t, :, None, :]).sum(3)
        dvv[:, t] = (r * k[:, t, :, :, None]).sum(2)
        dg[:, t] = (_carry(a[:, t], before) * r).sum((2, 3))
        r = _carry(a[:, t], r)

    def grouped(x):
        return x.reshape(batch, seqlen, groups, heads // groups, dk).sum(3)

    return dict(dq=grouped(dq), dk=grouped(dkk), dv=dvv, drate=-(step * dg).sum((0, 1)), dstep=-rate.double() * dg, dh0=r, dg=dg)


def _magnitude(x):
    return None if x is None else x.abs()


def everything(d, dy=None, dlast=None, scale=1.0, io=torch.float32):
    """{output: (value, bound)} for inputs d (q, k, v, rate, step, reset, h0)."""
    heads, dv = d["v"].shape[2:]
    seqlen, dk = d["q"].shape[1], d["q"].shape[3]
    m = dict(d, q=d["q"].abs(), k=d["k"].abs(), v=d["v"].abs(), h0=_magnitude(d.get("h0")))
    y, last, states = forward(scale=scale, **d)
    my, mlast, mstates = forward(scale=abs(scale), **m)
    n = 2 * (seqlen + dk + dv) + 160
    part = n * U
    rounded = 2 * HALF[io] if io == torch.bfloat16 else 0.0
    out = dict(y=(y, (part + rounded) * my + HALF[io] * y.abs()), last_state=(last, part * mlast))
    if dy is None:
        return out
    g = backward(dy=dy, dlast=dlast, scale=scale, states=states, **d)
    mg = backward(dy=dy.abs(), dlast=_magnitude(dlast), scale=abs(scale), states=mstates, **m)
    # dL/dg: sums of q . dq - k . dk over at most 512 tokens, of which all but what a_t <S, R> says cancels
    block = 512
    swing = (mg["dq"] * m["q"].double() + mg["dk"] * m["k"].double()).sum(3)       # [batch, seqlen, groups]
    swing = swing.repeat_interleave(heads // swing.shape[2], 2)
    pad = -seqlen % block
    swing = torch.nn.functional.pad(swing, (0, 0, 0, pad)).reshape(swing.shape[0], -1, block, heads)
    behind = swing.flip(2).cumsum(2).flip(2).reshape(swing.shape[0], -1, heads)[:, :seqlen]
    step = torch.ones_like(behind) if d.get("step") is None else d["step"].double()
    dg_bound = part * (behind + mg["dg"])
    for name in ("dq", "dk", "dv"):
        out[name] = (g[name], (part + rounded) * mg[name] + HALF[io] * g[name].abs())
    out["dh0"] = (g["dh0"], part * mg["dh0"])
    out["drate"] = (g["drate"], (step * dg_bound).sum((0, 1)) + U * g["drate"].abs())
    out["dstep"] = (g["dstep"], d["rate"].double() * dg_bound + HALF[io] * g["dstep"].abs())
    return out
