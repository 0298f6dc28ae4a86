"""The gated recurrence at the ends of its ranges, through the C ABI against the
token-by-token float64 form (needs an MI355X): states near the largest float,
gates far from their bias, batches of many short rows, memories of thousands of
tokens.

Bounds as in test_gated_gpu.py; what a case adds to them stands at the case.
"""
import numpy as np
import pytest
import torch

import gated_reference as ref
import selective_state_space_65_amd as ssm
from test_gated_gpu import DEV, IO, MODES, check, host, np64, run_all, say

pytestmark = pytest.mark.gpu


def normal(shape, seed, io="f32"):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(IO[io]).to(DEV)


def spike(L, seed):
    """Rows of one large token, 8 to 10 closed gates (a about 2e-9) after it and open ones before and behind: x, gate and
    the spikes' places, which run through a lane's tokens and across its end.  v stays within the 16 that the bounds of
    the gate's argument are derived for; the closed gates' own, at 20 to 23, is off by 32 u at most, and the state
    is gone after 5 of them, within K1 = 300 u."""
    dim = 12
    x, gate = normal((2, dim, L), seed), normal((2, dim, L), seed + 1).clamp(-3, 3) + 1.0
    at = [min(t, L - 1) for t in (0, 1, 2, 3, 5, 7, 8, 9, 13, L // 2, L // 2 + 1, L // 3)]
    for c, t in enumerate(at):
        gate[:, c, t + 1:t + 9 + c % 3] = -20.0 - (c % 4)
    return x, gate, at


@pytest.mark.parametrize("size", [1e34, -3e38])
@pytest.mark.parametrize("L", [7, 24, 60, 120, 250, 700, 3000, 9000])
def test_a_large_state_ends_at_closed_gates(L, size):
    """A state near the largest float is gone behind gates whose product is below every float.  A product of gates is
    rounded to a subnormal, or kept at the smallest, at most 16 times on its way to a token (8 factors of a chunk, 6 levels
    of lanes): 16 * 2^-149 of the state's size beside the bound of the arithmetic."""
    say("gated large state %g L=%d" % (size, L))
    x, gate, at = spike(L, 40 + L)
    for c, t in enumerate(at):
        x[:, c, t] = size
    y, last, ck = ssm.gated_scan_fwd_save(x, gate)
    torch.cuda.synchronize()
    f = ref.forward(np64(x), np64(gate))
    lost = 16 * 2.0 ** -149 * abs(size)
    check(y, f["y"], f["y_err"] + lost, "f32", "y")
    check(last, f["last"], f["last_err"] + lost, "f32", "last_state")


@pytest.mark.parametrize("size", [1e34, -3e37])
@pytest.mark.parametrize("L", [24, 60, 120, 250, 700, 3000])
def test_a_large_gradient_ends_at_closed_gates(L, size):
    """The same for the adjoint, against time: the large dy stands behind the closed gates, mirrored."""
    say("gated large gradient %g L=%d" % (size, L))
    x, gate, at = spike(L, 50 + L)
    dy = normal(x.shape, 60 + L)
    for c, t in enumerate(at):
        dy[:, c, t] = size
    gate, dy = gate.flip(-1).contiguous(), dy.flip(-1).contiguous()  # closed gates in front of the large token
    h0 = normal(x.shape[:2], 70)
    _, _, ck = ssm.gated_scan_fwd_save(x, gate, h0=h0)
    g = ssm.gated_scan_bwd(x, gate, dy, ck)
    torch.cuda.synchronize()
    b = ref.backward(np64(x), np64(gate), np64(dy), h0=np64(h0))
    f = ref.forward(np64(x), np64(gate), h0=np64(h0))
    a, _, da, _, _ = ref.gates(np64(gate), None, None, "plain")
    lost = 16 * 2.0 ** -149 * abs(size)
    hb = np.concatenate([np.abs(np64(h0))[..., None], f["bars"][..., :-1]], -1)
    check(g["dx"], b["dx"], b["dx_err"] + lost, "f32", "dx")
    check(g["dgate"], b["dgate"], b["dgate_err"] + lost * hb * da, "f32", "dgate")
    check(g["dh0"], b["dh0"], b["dh0_err"] + lost, "f32", "dh0")


@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [5, 40, 120, 600])
def test_a_bias_that_the_gate_cancels(L, mode, io, rate):
    """Biases up to 60 on either side and gates that bring their sum back to [-3, 3], so that memories stay within 100
    tokens.  Beside the bounds' 16 u for the argument: log2 e as a float is off by 1.4e-8, 63 * 1.4e-8 < 15 u, which K1 =
    300 u holds with 2 * 20 for the memory of sigmoid(3) (with a rate of 1.5 to 3, at least 0.07 off 1: 15 tokens)."""
    say("gated bias %s %s rate=%s L=%d" % (mode, io, rate, L))
    bias = torch.tensor([19.0, -19.5, 21.0, -20.5, 33.3, -27.7, 60.0, -59.0, 7.25])
    d = dict(x=normal((2, 9, L), 80, io), z=normal((2, 9, L), 81, io), h0=normal((2, 9), 82), reset=None,
             gate=(normal((2, 9, L), 83).clamp(-2.5, 2.5).cpu() - bias[:, None]).to(IO[io]).to(DEV),
             gate_bias=bias.to(DEV), rate=torch.linspace(1.5, 3.0, 9).to(DEV) if rate else None)
    run_all(d, io, mode, L, "bias")


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [6, 40, 120, 250, 700])
def test_a_gate_far_beyond_its_bias(L, mode):
    """Gates of -92 and 95 under biases of 20 and -20: v = -72 and 75, where sigmoid(v) and its distance from 1 are still
    normal floats, take a state of 1e31 to a number of the size of x and a token of 1e33 into it.  The argument of the
    exponential, about 110, is rounded by 44 u, and log2 e adds 20 u: twice that and the memory of 20 stay within K1."""
    say("gated far gate %s L=%d" % (mode, L))
    bias = torch.tensor([20.0, -20.0, 19.0, -19.0, 20.0, -20.0, 0.0])
    gate = normal((2, 7, L), 90).clamp(-2.5, 2.5).cpu() - bias[:, None]
    x = normal((2, 7, L), 91).cpu()
    for c in (0, 2, 4):  # the state goes through a nearly closed gate
        x[:, c, c], gate[:, c, c + 1] = 1e31, -92.0
    for c in (1, 3, 5):  # the token goes through its own, nearly open, gate
        x[:, c, c], gate[:, c, c] = (1e33 if mode == "convex" else 1e16 if mode == "norm" else 1.0), 95.0
    d = dict(x=x.to(DEV), gate=gate.to(DEV), gate_bias=bias.to(DEV), rate=None, z=None, reset=None, h0=normal((2, 7), 92))
    run_all(d, "f32", mode, L, "far")
    state = d["h0"].clone()
    f = ref.forward(mode=mode, **host(d))
    for t in range(6):
        y = ssm.gated_state_update(state, d["x"][..., t].contiguous(), d["gate"][..., t].contiguous(), d["gate_bias"],
                                   mode=mode)
        check(y, f["y"][..., t], f["y_err"][..., t], "f32", "token %d" % t)


def test_a_bias_that_is_not_finite():
    """A bias of -Inf closes its channel (y = w x, the state dropped), one of Inf holds the state, NaN stays in its channel;
    beyond 2^14 the same by size."""
    bias = torch.tensor([-float("inf"), float("inf"), float("nan"), -1e5, 1e5, 3e38, -3e38, 0.0], device=DEV)
    x, gate, h0 = normal((1, 8, 300), 95), normal((1, 8, 300), 96), normal((1, 8), 97)
    y, last = ssm.gated_scan_fwd(x, gate, bias, h0=h0, mode="convex")
    torch.cuda.synchronize()
    for c in (0, 3, 6):
        assert torch.equal(y[0, c], x[0, c])
    for c in (1, 4, 5):
        assert torch.equal(last[0, c], h0[0, c])
    assert torch.isnan(y[0, 2]).all() and torch.isfinite(y[0, 7]).all()


@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("shape", [(65536, 4, 1), (5000, 33, 7), (4096, 64, 64), (300, 65, 20), (9, 70, 700)])
def test_sums_over_many_batch_rows(shape, rate):
    """dgate_bias and drate over batches that no block holds whole, every row alike, so that each addition of a chain would
    be rounded the same way: within the bound of a tree of additions, whatever the batch."""
    say("gated batch sums %s rate=%s" % (shape, rate))
    batch, dim, L = shape
    d = dict(x=normal((1, dim, L), 100), gate=normal((1, dim, L), 101).clamp(-3, 3), h0=normal((1, dim), 102), z=None)
    d = {k: v if v is None else v.expand(batch, *v.shape[1:]).contiguous() for k, v in d.items()}
    d.update(gate_bias=torch.zeros(dim, device=DEV), reset=None,
             rate=torch.linspace(1.2, 3.0, dim).to(DEV) if rate else None)
    dy = normal((1, dim, L), 103).expand(shape).contiguous()
    kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}
    _, _, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], **kw)
    g = ssm.gated_scan_bwd(d["x"], d["gate"], dy, ck, **kw)
    one = {k: v if v is None or k in ("gate_bias", "rate") else v[:1] for k, v in d.items()}
    b = ref.backward(dy=np64(dy[:1]), mode="plain", **host(one))
    for k in ("dgate_bias", "drate")[:1 + rate]:
        check(g[k], batch * b[k], batch * b[k + "_err"], "f32", k)


def memory_of(d):
    """What the reference's bounds grow by: they are (2 tau + 64) u, taken as 300 u for memories of tau <= 100 tokens; here tau
    is the longest of the case's own gates, and no more than the tokens there are."""
    a, _, _, _, _ = ref.gates(np64(d["gate"]), np64(d["gate_bias"]), np64(d["rate"]), "plain")
    return (2 * min(1 / (1 - a).min(), a.shape[-1]) + 64) / 300


@pytest.mark.parametrize("constant", [False, True])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("gates", ["tau 1000", "tau 10000", "rates"])
def test_long_memory(gates, mode, constant):
    """Memories of thousands of tokens: a bias of a or of 1 - a that every token shares adds up over tau tokens, so the gates
    of a row also run as one constant, whose rounding every token does share."""
    L, dim = 6000, 7
    say("gated long memory %s %s constant=%s" % (gates, mode, constant))
    # x of one sign: the states are as large as the sums of magnitudes that the bounds are taken of
    d = dict(x=normal((1, dim, L), 110).abs(), z=normal((1, dim, L), 111), h0=normal((1, dim), 112).abs(), reset=None, rate=None)
    gate = normal((1, dim, 1), 113).expand(1, dim, L) if constant else normal((1, dim, L), 113)
    d["gate"] = gate.clamp(-1, 1).contiguous()
    if gates == "rates":
        d.update(rate=torch.logspace(-2.7, -1, dim).to(DEV), gate_bias=normal((dim,), 114).clamp(-1, 1))
    else:
        tau = float(gates.split()[1])
        d["gate_bias"] = torch.full((dim,), float(np.log(tau - 1)), device=DEV)
    run_all(d, "f32", mode, 7, "long", memory=memory_of(d))
    # the decode step, from the state in the middle of the row
    f = ref.forward(mode=mode, **host(d))
    state = torch.tensor(f["states"][..., 2999], dtype=torch.float32, device=DEV)
    part = {k: d[k] if k in ("gate_bias", "rate") else None if d[k] is None else d[k][..., 3000:3200].contiguous()
            for k in ("x", "gate", "z", "gate_bias", "rate")}
    y = torch.stack([ssm.gated_state_update(state, *(part[k][..., t].contiguous() for k in ("x", "gate")),
                                            d["gate_bias"], d["rate"], part["z"][..., t].contiguous(), mode=mode)
                     for t in range(200)], -1)
    # the state taken over is rounded once; 200 tokens add 200 roundings of 2 u to the gates' 64 u
    check(y, f["y"][..., 3000:3200], f["y_err"][..., 3000:3200] * (2 * 200 + 65) / 300, "f32", "steps")
