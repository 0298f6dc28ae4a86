"""Calls of the gated recurrence and the norms as programs make them (needs an
MI355X): tensors in the wrong place beside a stream, and backwards that sum in
a workspace on other streams and in captured graphs.
"""
import ctypes

import pytest
import torch

import selective_state_space_65_amd as ssm
from selective_state_space_65_amd import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_host_tensors_beside_a_stream():
    """A tensor left on the host is refused by name, with a stream as without one."""
    x, state = torch.randn((2, 6, 300), device=DEV), torch.randn((2, 6), device=DEV)
    tok = x[..., 0].contiguous()
    _, _, ck = ssm.gated_scan_fwd_save(x, x)
    _, _, mean, rstd = ssm.norm_fwd(tok)
    side = torch.cuda.Stream()
    for stream in (None, side):
        for name, call in (("gate", lambda: ssm.gated_scan_fwd(x, x.cpu(), stream=stream)),
                           ("z", lambda: ssm.gated_scan_fwd_save(x, x, z=x.cpu(), stream=stream)),
                           ("dy", lambda: ssm.gated_scan_bwd(x, x, x.cpu(), ck, stream=stream)),
                           ("gate", lambda: ssm.gated_state_update(state, tok, tok.cpu(), stream=stream)),
                           ("residual", lambda: ssm.norm_fwd(tok, residual=tok.cpu(), stream=stream)),
                           ("rstd", lambda: ssm.norm_bwd(tok, tok, rstd.cpu(), mean=mean, stream=stream))):
            with pytest.raises(ValueError, match=name + ": expected device"):
                call()
    torch.cuda.synchronize()


# Batches that no block of the backward holds whole: a row of 3 and of 2 waves, of 16 lanes and of 64.
SUMMED = [(3, 300, 1500), (9, 200, 900), (17, 130, 100), (9, 64, 300)]


def training_call(shape, seed, stream=None):
    g = torch.Generator().manual_seed(seed)
    x, gate, dy = (torch.randn(shape, generator=g).to(DEV, torch.bfloat16) for _ in range(3))
    rate = torch.rand(shape[1], generator=g).to(DEV) + 0.1
    bias = torch.randn(shape[1], generator=g).to(DEV)
    torch.cuda.synchronize()

    def call():
        _, _, ck = ssm.gated_scan_fwd_save(x, gate, bias, rate, stream=stream)
        return ssm.gated_scan_bwd(x, gate, dy, ck, bias, rate, stream=stream)

    return call


def same(a, b):
    return all(torch.equal(a[k], b[k]) for k in ("dx", "dgate", "dgate_bias", "drate", "dh0"))


def test_the_shapes_below_sum_in_a_workspace():
    n = ctypes.c_int64(0)
    for shape in SUMMED:
        assert binding.load_library().ssm_gated_scan_bwd_workspace_bytes(*shape, 1, ctypes.byref(n)) == 0
        assert n.value == 2 * shape[0] * shape[1] * 4, shape


@pytest.mark.parametrize("shape", SUMMED)
def test_workspace_on_another_stream(shape):
    """stream=: partial sums and their reduction are ordered on that stream, and the workspace's memory is not handed to
    the current stream before they are done."""
    print("[gpu-case] workspace on another stream %s" % (shape,), flush=True)
    want = training_call(shape, 1)()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    call = training_call(shape, 1, side)
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        got = call()
        torch.empty(2 * shape[0] * shape[1] * 4, dtype=torch.uint8, device=DEV).fill_(255)
        torch.cuda.current_stream().wait_stream(side)
        assert same(got, want)


def test_workspaces_on_two_streams_at_once():
    """Backwards of changing sizes on two streams, never the same size on both at a time."""
    print("[gpu-case] workspaces on two streams", flush=True)
    calls = [training_call(s, 2 + i) for i, s in enumerate(SUMMED)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for k in range(24):
        for i, s in enumerate(streams):
            j = (k + 2 * i) % len(calls)
            with torch.cuda.stream(s):
                got.append((j, calls[j]()))
    torch.cuda.synchronize()
    for j, g in got:
        assert same(g, want[j]), SUMMED[j]


def test_workspaces_in_two_graphs():
    """Two captured backwards of different sizes on one memory pool, replayed in turn with eager ones between: the gradients
    of each replay are read before the next may write its own."""
    calls = [training_call(s, 20 + i) for i, s in enumerate(SUMMED[:2])]
    want = [c() for c in calls]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graphs, pool = [], None
    for c in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool, stream=side):
            held = c()
        pool = g.pool()
        graphs.append((g, held))
    for k in range(6):
        g, held = graphs[k % 2]
        print("[gpu-case] workspace graph replay %d" % k, flush=True)
        g.replay()
        torch.cuda.synchronize()
        assert same(held, want[k % 2])
        assert same(calls[1 - k % 2](), want[1 - k % 2])
        torch.cuda.synchronize()
