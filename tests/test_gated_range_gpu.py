"""The gated recurrence at the ends of its ranges, through the C ABI against the
token-by-token float64 form (needs an MI355X): states near the largest float.

Bounds as in test_gated_gpu.py; what a case adds to them stands at the case.
"""
import numpy as np
import pytest
import torch

import gated_reference as ref
import selective_state_space_65_amd as ssm
from test_gated_gpu import DEV, IO, MODES, check, host, np64, say

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
