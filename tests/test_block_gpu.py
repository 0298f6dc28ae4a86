"""The norm and the gated recurrence together, as a block uses them (needs an
MI355X): residual stream -> norm -> projections -> recurrence -> projection ->
residual add of the next norm.  A training step against float64 autograd, a
prompt continued token by token against the whole sequence, the recurrence
beside the selective scan on the same normed input, and a decode step of the
block in captured graphs.

The block's products are torch's.  Bars are the ones the library's scans are
held to: 1e-4 of an output's largest magnitude in fp32, 2e-2 in bf16.
"""
import numpy as np
import pytest
import torch

import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BAR = {torch.float32: 1e-4, torch.bfloat16: 2e-2}


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def weights(d, dim, io, seed, layers=2):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(layers):
        out.append(dict(w=1 + 0.1 * torch.randn(d, generator=g), b=0.1 * torch.randn(d, generator=g),
                        win=torch.randn(3 * dim, d, generator=g) * d ** -0.5,
                        wout=torch.randn(d, dim, generator=g) * dim ** -0.5,
                        gate_bias=torch.empty(dim).uniform_(0.0, 3.0, generator=g),
                        rate=torch.empty(dim).uniform_(0.1, 2.0, generator=g)))
    return [{k: v.to(DEV, io if k in ("win", "wout") else torch.float32) for k, v in p.items()} for p in out]


def project(w, n):
    """(batch, seqlen, d) -> (batch, rows of w, seqlen), contiguous."""
    return torch.matmul(w, n.transpose(1, 2).contiguous())


def forward(x, layers, reset, mode, state=None):
    """Returns the last sum and, for each layer, what its backward needs; states are carried in place when given."""
    res, saved, dim = None, [], layers[0]["wout"].shape[1]
    for i, p in enumerate(layers):
        n, s, mean, rstd = ssm.norm_fwd(x, weight=p["w"], bias=p["b"], residual=res)
        v = project(p["win"], n)
        u, gate, z = (t.contiguous() for t in v.split(dim, 1))
        h0 = None if state is None else state[i]
        y, last, ck = ssm.gated_scan_fwd_save(u, gate, p["gate_bias"], p["rate"], z, reset, h0, mode, last_state=h0)
        x = torch.matmul(y.transpose(1, 2).contiguous(), p["wout"].t())
        res = s
        saved.append((n, s, mean, rstd, u, gate, z, y, ck))
    return x, res, saved


def backward(dx, dres, layers, saved, reset, mode):
    """Gradients of x and of each layer's parameters, given those of the last layer's output and sum."""
    grads = []
    for p, (n, s, mean, rstd, u, gate, z, y, ck) in reversed(list(zip(layers, saved))):
        yt = y.transpose(1, 2).contiguous()
        dwout = torch.matmul(dx.flatten(0, 1).t().contiguous(), yt.flatten(0, 1))
        dy = torch.matmul(dx, p["wout"]).transpose(1, 2).contiguous()
        g = ssm.gated_scan_bwd(u, gate, dy, ck, p["gate_bias"], p["rate"], z, reset, mode=mode)
        dv = torch.cat([g["dx"], g["dgate"], g["dz"]], 1)
        dvt = dv.transpose(1, 2).contiguous()
        dwin = torch.matmul(dvt.flatten(0, 1).t().contiguous(), n.flatten(0, 1))
        dn = torch.matmul(dvt, p["win"])
        gn = ssm.norm_bwd(dn, s, rstd, mean=mean, weight=p["w"], dresidual_out=dres)
        grads.append(dict(w=gn["dweight"], b=gn["dbias"], win=dwin, wout=dwout, gate_bias=g["dgate_bias"],
                          rate=g["drate"]))
        dx, dres = gn["dx"], gn["dresidual"] if gn["dresidual"] is not None else gn["dx"]
    return dx, grads[::-1]


def reference(x, layers, reset, mode):
    """The same block in float64 on the CPU, for autograd."""
    res, dim = None, layers[0]["wout"].shape[1]
    for p in layers:
        s = x if res is None else x + res
        c = s - s.mean(-1, keepdim=True)
        n = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * p["w"] + p["b"]
        u, gate, z = torch.einsum("ed,bld->bel", p["win"], n).split(dim, 1)
        a = torch.exp(-p["rate"][:, None] * torch.sigmoid(gate + p["gate_bias"][:, None]))
        w = {"plain": torch.ones_like(a), "convex": 1 - a, "norm": torch.sqrt(1 - a * a)}[mode]
        keep = a * (reset == 0).double()[:, None, :]
        h, hs = torch.zeros_like(u[..., 0]), []
        for t in range(u.shape[2]):
            h = keep[..., t] * h + w[..., t] * u[..., t]
            hs.append(h)
        y = torch.stack(hs, -1) * torch.nn.functional.silu(z)
        x, res = torch.einsum("bel,de->bld", y, p["wout"]), s
    return x, res


def close(got, want, bar, what):
    got, want = got.double().cpu(), want.detach().double().cpu()
    err, scale = (got - want).abs().max().item(), want.abs().max().item()
    assert err <= bar * scale, "%s: %.3g of its largest magnitude" % (what, err / scale)


@pytest.mark.parametrize("mode", ["plain", "convex", "norm"])
@pytest.mark.parametrize("shape", [(2, 37, 24, 40), (3, 300, 65, 33)])
def test_training_step(shape, mode):
    """Two layers, packed sequences, fp32: outputs and every gradient against autograd."""
    batch, L, d, dim = shape
    say("block training step %s %s" % (shape, mode))
    layers = weights(d, dim, torch.float32, 3)
    g = torch.Generator().manual_seed(4)
    x = torch.randn((batch, L, d), generator=g).to(DEV)
    reset = (torch.rand((batch, L), generator=g) < 0.05).to(torch.uint8).to(DEV)
    do, ds = torch.randn((batch, L, d), generator=g).to(DEV), torch.randn((batch, L, d), generator=g).to(DEV)
    out, res, saved = forward(x, layers, reset, mode)
    dx, grads = backward(do, ds, layers, saved, reset, mode)
    torch.cuda.synchronize()
    xr = x.double().cpu().requires_grad_()
    lr = [{k: v.double().cpu().requires_grad_() for k, v in p.items()} for p in layers]
    o, r = reference(xr, lr, reset.cpu(), mode)
    ((o * do.double().cpu()).sum() + (r * ds.double().cpu()).sum()).backward()
    close(out, o, 1e-4, "output")
    close(res, r, 1e-4, "sum")
    close(dx, xr.grad, 1e-4, "dx")
    for i, (got, want) in enumerate(zip(grads, lr)):
        for k in want:
            close(got[k], want[k].grad, 1e-4, "layer %d d%s" % (i, k))


def decode(x, layers, states, mode):
    """One token (batch, d) through the layers; the states move on in place."""
    res, dim = None, layers[0]["wout"].shape[1]
    for p, h in zip(layers, states):
        n, s, _, _ = ssm.norm_fwd(x, weight=p["w"], bias=p["b"], residual=res, save_stats=False)
        u, gate, z = (t.contiguous() for t in torch.matmul(n, p["win"].t()).split(dim, 1))
        y = ssm.gated_state_update(h, u, gate, p["gate_bias"], p["rate"], z, mode=mode)
        x, res = torch.matmul(y, p["wout"].t()), s
    return x + res


@pytest.mark.parametrize("io", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens(io):
    """A prompt, then token by token from its states, equals the whole sequence at once."""
    batch, L, cut, d, dim = 3, 140, 131, 64, 96
    layers = weights(d, dim, io, 5)
    x = torch.randn((batch, L, d), generator=torch.Generator().manual_seed(6)).to(DEV, io)
    reset = torch.zeros((batch, L), dtype=torch.uint8, device=DEV)
    whole, res, _ = forward(x, layers, reset, "norm")
    whole = whole + res
    states = [torch.zeros((batch, dim), device=DEV) for _ in layers]
    forward(x[:, :cut].contiguous(), layers, reset[:, :cut].contiguous(), "norm", states)
    for t in range(cut, L):
        close(decode(x[:, t].contiguous(), layers, states, "norm"), whole[:, t], BAR[io], "token %d" % t)


def test_beside_the_selective_scan():
    """The normed input feeds the selective scan and the recurrence in one layer; with dstate 1, B = C = 1 and A = -1 the
    selective scan is the plain recurrence of a = exp(-softplus(delta)), which the gate -delta gives: both agree."""
    batch, dim, L = 2, 70, 520
    s = torch.randn((batch, L, dim), generator=torch.Generator().manual_seed(7)).to(DEV)
    n = ssm.norm_fwd(s, kind="rms")[0].transpose(1, 2).contiguous()
    delta = 0.5 * torch.randn((batch, dim, L), generator=torch.Generator().manual_seed(8)).to(DEV) - 2.0
    one = torch.ones((batch, 1, L), device=DEV)
    y, last = ssm.scan_fwd(n, delta, torch.full((dim, 1), -1.0, device=DEV), one, one, delta_softplus=True)
    x = n * torch.nn.functional.softplus(delta)       # the scan's input term, Delta u
    y2, last2 = ssm.gated_scan_fwd(x, -delta)         # exp(-softplus(delta)) = sigmoid(-delta)
    close(y2, y, 1e-4, "y")
    close(last2, last[..., 0], 1e-4, "last_state")


def test_decode_graphs_share_states_and_memory():
    """Two graphs of the block's decode step on one memory pool, replayed in turn with eager work between."""
    batch, d, dim = 4, 48, 80
    layers = weights(d, dim, torch.bfloat16, 9)
    x = torch.randn((batch, d), device=DEV).bfloat16()
    states = [torch.zeros((batch, dim), device=DEV) for _ in layers]
    eager = [h.clone() for h in states]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode(x, layers, [h.clone() for h in states], "convex")
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs, pool = [], None
    for mode in ("convex", "norm"):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool, stream=side):
            out = decode(x, layers, states, mode)
        pool = g.pool()
        graphs.append((mode, g, out))
    for i in range(6):
        mode, g, out = graphs[i % 2]
        say("block decode graph %s replay %d" % (mode, i))
        x.copy_(torch.randn((batch, d), device=DEV))
        want = decode(x, layers, eager, mode)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        for h, e in zip(states, eager):
            assert torch.equal(h, e)
        _ = float(np.float64(out.float().abs().sum().item()))


def test_two_streams_at_once():
    """Norms and recurrences of different sizes on two streams at the same time give what they give alone."""
    g = torch.Generator().manual_seed(11)
    jobs = []
    for batch, dim, L, io in ((3, 200, 700, torch.bfloat16), (5, 130, 90, torch.float32)):
        x = [torch.randn((batch, dim, L), generator=g).to(DEV, io) for _ in range(4)]
        r = torch.randn((batch * 40, dim), generator=g).to(DEV, io)
        jobs.append((x, r))

    def call(x, r):
        y, last, ck = ssm.gated_scan_fwd_save(x[0], x[1], z=x[2], mode="norm")
        gr = ssm.gated_scan_bwd(x[0], x[1], x[3], ck, z=x[2], mode="norm")
        n, s, mean, rstd = ssm.norm_fwd(r)
        gn = ssm.norm_bwd(n, s, rstd, mean=mean)
        return [y, last, *(v for v in gr.values() if v is not None), n, *(v for v in gn.values() if v is not None)]

    want = [call(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for u, v in zip(run, want[i]):
                assert torch.equal(u, v)
