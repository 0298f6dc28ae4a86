"""The gated recurrence (forward, backward, decode step) through the C ABI
against the token-by-token float64 form (needs an MI355X).

Every output value is held to its own bound: the fp32 arithmetic's
(gated_reference) plus, for an io output, half a step of its type (2^-8
relative in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest
import torch

import gated_reference as ref
import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
IO = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
MODES = ["plain", "convex", "norm"]


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def draw(batch, dim, L, io, seed, rate=False, z=True, reset=True, h0=True):
    """Inputs as device tensors, in the value ranges the bounds are derived for: memory of at most 100 tokens."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng([seed, 1])

    def normal(*shape):
        return torch.randn(shape, generator=g)

    d = dict(x=normal(batch, dim, L).to(IO[io]), gate=normal(batch, dim, L).clamp(-3, 3).to(IO[io]))
    if rate:  # a >= exp(-rate), 1 - a >= rate * sigmoid(-4) / 2
        d["rate"] = torch.tensor(r.uniform(1.2, 4.0, dim), dtype=torch.float32)
        d["gate_bias"] = torch.tensor(r.uniform(-1.0, 1.0, dim), dtype=torch.float32)
    else:
        d["rate"] = None
        d["gate_bias"] = torch.tensor(r.uniform(-2.0, 1.5, dim), dtype=torch.float32)
    d["z"] = normal(batch, dim, L).to(IO[io]) if z else None
    d["reset"] = (torch.rand((batch, L), generator=g) < 0.03).to(torch.uint8) if reset else None
    d["h0"] = normal(batch, dim) if h0 else None
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def host(d):
    return {k: np64(v) for k, v in d.items()}


def check(got, want, err, io, what):
    got = np64(got)
    assert got.shape == want.shape, what
    bound = err * (1 + HALF[io]) + HALF[io] * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound, at %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / bound), np.argwhere(bad)[0])


def run_all(d, io, mode, seed, what, dlast=True, memory=1.0):
    """Forward with checkpoints, backward; both against the reference.  memory: the longest memory over the 100 tokens
    the reference's bounds assume, which they grow with."""
    batch, dim, L = d["x"].shape
    g = torch.Generator().manual_seed(seed + 1000)
    dy = torch.randn((batch, dim, L), generator=g).to(IO[io]).to(DEV)
    dl = torch.randn((batch, dim), generator=g).to(DEV) if dlast else None
    kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}
    y, last, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], mode=mode, **kw)
    gr = ssm.gated_scan_bwd(d["x"], d["gate"], dy, ck, dlast=dl, mode=mode, **kw)
    torch.cuda.synchronize()
    h = host(d)
    f = ref.forward(mode=mode, **h)
    b = ref.backward(dy=np64(dy), dlast=np64(dl), mode=mode, **h)
    for r in (f, b):
        r.update({k: v * memory for k, v in r.items() if k.endswith("_err")})
    check(y, f["y"], f["y_err"], io, what + " y")
    check(last, f["last"], f["last_err"], "f32", what + " last_state")
    for i in range(ck.shape[2]):
        want = (f["states"][..., 128 * i - 1] if i else (h["h0"] if h["h0"] is not None else np.zeros((batch, dim))))
        bar = f["bars"][..., 128 * i - 1] if i else np.abs(want)
        check(ck[..., i], want, memory * ref.K1 * bar, "f32", what + " ckpt")
    for k in ("dx", "dgate", "dz"):
        if k in b:
            check(gr[k], b[k], b[k + "_err"], io, what + " " + k)
        else:
            assert gr[k] is None
    for k in ("dgate_bias", "drate", "dh0"):
        if k in b:
            check(gr[k], b[k], b[k + "_err"], "f32", what + " " + k)
        else:
            assert gr[k] is None
    return y, last, ck, gr


# One token; inside and on the edges of a lane (8), of 8 lanes (64), of 16
# lanes (128), of a wave (512) and of a block's waves; channel counts that leave
# the last wave or block part empty; batch rows that fit one block of the
# backward and that do not, at one wave a row and at several.
SHAPES = [(1, 1, 1), (3, 70, 1), (2, 33, 5), (2, 65, 8), (1, 3, 9), (2, 37, 31), (5, 9, 64), (1, 17, 65), (2, 5, 100),
          (3, 7, 128), (1, 2, 129), (2, 3, 511), (1, 3, 512), (2, 2, 513), (1, 5, 1000), (2, 1, 1024), (1, 2, 1025),
          (1, 2, 4099), (1, 1, 9001), (2, 4100, 131), (1, 8200, 160), (8, 3, 300), (9, 2, 300), (4, 5, 600), (5, 4, 1030),
          (2, 2, 2100), (3, 2, 1500), (17, 1, 4000), (8, 3, 200), (9, 3, 200), (7, 40, 250), (16, 5, 100), (17, 5, 100),
          (32, 3, 50), (33, 2, 50), (5, 37, 60), (256, 2, 7), (257, 2, 7), (3, 200, 4), (4, 9000, 140)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, io):
    i = SHAPES.index(shape)
    mode, rate = MODES[i % 3], (i // 3) % 2 == 1
    say("gated %s %s %s rate=%s" % (shape, io, mode, rate))
    run_all(draw(*shape, io, 70 + i, rate=rate, z=i % 2 == 0, reset=i % 4 != 3, h0=i % 5 != 4), io, mode, i,
            "%s %s" % (shape, io))


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [6, 40, 120, 700])
def test_modes_and_options(mode, rate, io, L):
    """Each kernel variant with every option on, and with none."""
    say("gated options %s rate=%s %s L=%d" % (mode, rate, io, L))
    run_all(draw(2, 9, L, io, 300 + L, rate=rate), io, mode, L, "all on")
    d = draw(2, 9, L, io, 301 + L, rate=rate, z=False, reset=False, h0=False)
    d["gate_bias"] = None
    run_all(d, io, mode, L, "all off", dlast=False)


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [1, 7, 50, 120, 250, 700, 1500])
def test_rates_around_a_quarter(L, mode, io):
    """Rates below 1/4 (1 - a from its series alone), on it and above it, in every lane or side by side: v >= -4, so 1 - a is
    at least 0.15 * 0.018 / 1.02 and a token's memory at most 380 tokens."""
    for k in range(3):
        d = draw(2, 13, L, io, 1700 + k, rate=True)
        rate = torch.linspace(0.15, 0.249, 13)
        if k:
            rate[5], rate[9] = 0.25, 0.26
        if k == 2:
            rate[::2] = 3.0
        d["rate"] = rate.to(DEV)
        run_all(d, io, mode, L, "rates %d" % k, memory=3.8)


@pytest.mark.parametrize("L", [5, 60, 128, 2000])
def test_rows_of_resets(L):
    """A row with a reset at every token, one with none, one with the first token only: h = w x in the first."""
    d = draw(3, 6, L, "f32", 400 + L)
    d["reset"].zero_()
    d["reset"][0] = 255
    d["reset"][2, 0] = 1
    y, _, _, g = run_all(d, "f32", "convex", 5, "resets")
    assert g["dh0"][0].abs().max() == 0 and g["dh0"][2].abs().max() == 0
    again = ssm.gated_scan_fwd(d["x"], d["gate"], d["gate_bias"], z=d["z"], reset=d["reset"].bool(), h0=d["h0"],
                               mode="convex")[0]
    assert torch.equal(y, again)


@pytest.mark.parametrize("L", [7, 50, 128, 1500, 5000])
@pytest.mark.parametrize("poison", [float("inf"), float("nan")])
def test_reset_stops_what_is_not_finite(L, poison):
    """Infinities and NaN in x before a reset, and in the initial state, reach no token after it, and in the
    backward nothing before the reset takes a gradient from after it."""
    say("gated poison %s L=%d" % (poison, L))
    d = draw(2, 5, L, "f32", 500 + L)
    cut = L // 2
    d["reset"].zero_()
    d["reset"][:, cut] = 1
    clean = ssm.gated_scan_fwd(d["x"], d["gate"], d["gate_bias"], z=d["z"], reset=d["reset"], h0=d["h0"], mode="norm")
    bad = dict(d, x=d["x"].clone(), h0=torch.full_like(d["h0"], poison))
    bad["x"][:, :, 0] = poison
    y, last, ck = ssm.gated_scan_fwd_save(bad["x"], bad["gate"], d["gate_bias"], z=d["z"], reset=d["reset"],
                                          h0=bad["h0"], mode="norm")
    torch.cuda.synchronize()
    # within the rounding of another combination order: the tiles before the cut run either way
    assert torch.isfinite(y[:, :, cut:]).all() and torch.isfinite(last).all()
    assert torch.allclose(y[:, :, cut:], clean[0][:, :, cut:], rtol=1e-5, atol=1e-6)
    assert not torch.isfinite(y[:, :, 0]).any()
    dy = torch.ones_like(d["x"])
    dy[:, :, L - 1] = poison
    g = ssm.gated_scan_bwd(d["x"], d["gate"], dy, ssm.gated_scan_fwd_save(d["x"], d["gate"], d["gate_bias"], z=d["z"],
                           reset=d["reset"], h0=d["h0"], mode="norm")[2], d["gate_bias"], z=d["z"], reset=d["reset"],
                           mode="norm")
    torch.cuda.synchronize()
    assert torch.isfinite(g["dx"][:, :, :cut]).all() and torch.isfinite(g["dgate"][:, :, :cut]).all()
    assert torch.isfinite(g["dh0"]).all()
    assert not torch.isfinite(g["dx"][:, :, L - 1]).any()


@pytest.mark.parametrize("L", [100, 1000, 3000])
def test_infinity_propagates(L):
    """Without a reset an infinite state stays infinite through products of gates far below the smallest float."""
    d = draw(1, 4, L, "f32", 600, z=False, reset=False)
    d["gate_bias"] = torch.full((4,), -20.0, device=DEV)  # a about 2e-9: the product underflows within 5 tokens
    d["x"][0, 1, 3] = float("inf")
    y, last = ssm.gated_scan_fwd(d["x"], d["gate"], d["gate_bias"], h0=d["h0"])
    torch.cuda.synchronize()
    assert torch.isinf(y[0, 1, 3:]).all() and torch.isinf(last[0, 1])
    assert torch.isfinite(y[0, 1, :3]).all() and torch.isfinite(y[0, [0, 2, 3]]).all()


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [6, 60, 120, 200, 1100, 4100])
def test_nan_gate_propagates(mode, L):
    """A NaN gate makes every later state of its channel NaN, wherever it stands in a lane's tokens, until a reset; in the
    backward it reaches every earlier token."""
    d = draw(1, 12, L, "f32", 650, z=False)
    d["reset"].zero_()
    at = [0, 1, 2, 3, 4, 5, L // 2, L // 2 + 1, L - 2, L - 1]
    for c, t in enumerate(at):
        d["gate"][0, c, t] = float("nan")
    d["gate"][0, 10, 0] = float("nan")
    y, last, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], d["gate_bias"], h0=d["h0"], mode=mode)
    g = ssm.gated_scan_bwd(d["x"], d["gate"], d["x"], ck, d["gate_bias"], mode=mode)
    torch.cuda.synchronize()
    for c, t in enumerate(at):
        assert torch.isfinite(y[0, c, :t]).all() and torch.isnan(y[0, c, t:]).all() and torch.isnan(last[0, c]), (c, t)
        assert torch.isnan(g["dx"][0, c, :t]).all() and torch.isfinite(g["dx"][0, c, t + 1:]).all(), (c, t)
        assert torch.isnan(g["dh0"][0, c])
    assert torch.isfinite(y[0, 11]).all() and torch.isfinite(g["dx"][0, 11]).all()
    d["reset"][0, L // 2] = 1
    y = ssm.gated_scan_fwd(d["x"], d["gate"], d["gate_bias"], reset=d["reset"], h0=d["h0"], mode=mode)[0]
    assert torch.isnan(y[0, 10, :L // 2]).all() and torch.isfinite(y[0, 10, L // 2:]).all()


@pytest.mark.parametrize("rate", [False, True])
@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("L", [4, 61, 127, 900])
def test_extreme_gates(mode, rate, L):
    """Gates at -inf, +inf and the type's extremes: a is 0 or 1 exactly, w its limit, and no output or gradient is NaN."""
    d = draw(2, 6, L, "bf16", 700 + L, rate=rate)
    lo, hi = torch.finfo(torch.bfloat16).min, torch.finfo(torch.bfloat16).max
    d["gate"][0, 0], d["gate"][0, 1], d["gate"][0, 2], d["gate"][0, 3] = -float("inf"), float("inf"), lo, hi
    d["gate"][1, 4, ::2] = -float("inf")
    d["gate"][1, 5, 1::3] = float("inf")
    y, _, _, g = run_all(d, "bf16", mode, 11, "extreme")
    for k, v in g.items():
        assert v is None or torch.isfinite(v).all(), k
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("cuts", [(1, 2, 3), (8, 64, 100), (128, 512, 1300), (777,)])
def test_carried_state(cuts, io):
    """Pieces of a sequence, the state carried in place, equal the whole within the bounds."""
    L = 1501
    d = draw(2, 7, L, io, 800, rate=True)
    state = d["h0"].clone()
    edges = [0, *cuts, L]
    parts = []
    for a, b in zip(edges, edges[1:]):
        piece = {k: (d[k][..., a:b].contiguous() if d[k] is not None else None) for k in ("x", "gate", "z", "reset")}
        y, last = ssm.gated_scan_fwd(piece["x"], piece["gate"], d["gate_bias"], d["rate"], piece["z"], piece["reset"],
                                     h0=state, last_state=state, mode="norm")
        assert last is state
        parts.append(y)
    f = ref.forward(mode="norm", **host(d))
    check(torch.cat(parts, -1), f["y"], f["y_err"], io, "pieces")
    check(state, f["last"], f["last_err"], "f32", "state")


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [1, 5, 64, 252, 1000, 2561])
@pytest.mark.parametrize("rate", [False, True])
def test_step(dim, rate, io):
    """The decode step, three tokens in a row, against the reference."""
    i = [1, 5, 64, 252, 1000, 2561].index(dim)
    mode, batch, L = MODES[i % 3], 1 + i % 4, 3
    d = draw(batch, dim, L, io, 900 + i, rate=rate, z=i % 2 == 0, reset=False)
    state = d["h0"].clone()
    ys = []
    for t in range(L):
        tok = {k: None if d[k] is None else d[k][..., t].contiguous() for k in ("x", "gate", "z")}
        ys.append(ssm.gated_state_update(state, tok["x"], tok["gate"], d["gate_bias"], d["rate"], tok["z"], mode=mode))
    f = ref.forward(mode=mode, **host(d))
    check(torch.stack(ys, -1), f["y"], f["y_err"], io, "step")
    check(state, f["last"], f["last_err"], "f32", "state")
    one = {k: None if d[k] is None else d[k][..., :1].contiguous() for k in ("x", "gate", "z")}
    y1, l1 = ssm.gated_scan_fwd(one["x"], one["gate"], d["gate_bias"], d["rate"], one["z"], h0=d["h0"], mode=mode)
    s1 = d["h0"].clone()
    y2 = ssm.gated_state_update(s1, one["x"][..., 0].contiguous(), one["gate"][..., 0].contiguous(), d["gate_bias"],
                                d["rate"], None if one["z"] is None else one["z"][..., 0].contiguous(), mode=mode)
    assert torch.equal(y1[..., 0], y2) and torch.equal(l1, s1)


def framed(shape, dtype, offset, fill):
    """A contiguous tensor `offset` elements into a larger buffer filled with `fill`, and that buffer."""
    n = int(np.prod(shape))
    buf = torch.full((n + offset + 64,), fill, dtype=dtype, device=DEV)
    return buf[offset:offset + n].view(shape), buf


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 3, 6), (2, 5, 37), (1, 7, 125), (2, 3, 1029)])
@pytest.mark.parametrize("offset", [1, 3])
def test_any_alignment_and_nothing_else_written(shape, io, offset):
    """Inputs and outputs that start at any element: the same bits as from aligned ones, and no byte around an output changes."""
    d = draw(*shape, io, 1000, rate=True)
    dy = torch.randn(shape, generator=torch.Generator().manual_seed(3)).to(IO[io]).to(DEV)
    kw = {k: d[k] for k in ("gate_bias", "rate")}
    y, last, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], z=d["z"], reset=d["reset"], h0=d["h0"], mode="norm", **kw)
    g = ssm.gated_scan_bwd(d["x"], d["gate"], dy, ck, z=d["z"], reset=d["reset"], mode="norm", **kw)
    moved = {}
    for k, v in dict(d, dy=dy).items():
        if k in ("x", "gate", "z", "dy", "reset"):
            moved[k], _ = framed(v.shape, v.dtype, offset, 1)
            moved[k].copy_(v)
    out, ob = framed(shape, IO[io], offset, 7)
    l2, lb = framed(last.shape, torch.float32, offset, 7)
    c2, cb = framed(ck.shape, torch.float32, offset, 7)
    ssm.gated_scan_fwd(moved["x"], moved["gate"], z=moved["z"], reset=moved["reset"], h0=d["h0"], mode="norm", out=out,
                       last_state=l2, ckpt=c2, **kw)
    g2 = ssm.gated_scan_bwd(moved["x"], moved["gate"], moved["dy"], c2, z=moved["z"], reset=moved["reset"],
                            mode="norm", **kw)
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(l2, last) and torch.equal(c2, ck)
    for b, v in ((ob, out), (lb, l2), (cb, c2)):
        n = v.numel()
        assert (b[:offset] == 7).all() and (b[offset + n:] == 7).all()
    for k in g:
        assert torch.equal(g[k], g2[k]), k


def test_deterministic():
    d = draw(3, 200, 1500, "bf16", 1100, rate=True)
    a = run_twice(d)
    for u, v in zip(*a):
        assert torch.equal(u, v)


def run_twice(d):
    out = []
    for _ in range(2):
        kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}
        y, last, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], mode="norm", **kw)
        g = ssm.gated_scan_bwd(d["x"], d["gate"], d["z"], ck, mode="norm", **kw)
        out.append([y, last, ck, *g.values()])
    return out


def test_need_selects_outputs():
    d = draw(2, 10, 300, "f32", 1200, rate=True)
    kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}
    _, _, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], **kw)
    full = ssm.gated_scan_bwd(d["x"], d["gate"], d["x"], ck, **kw)
    for name in ("dgate_bias", "drate", "dz", "dh0"):
        g = ssm.gated_scan_bwd(d["x"], d["gate"], d["x"], ck, need=(name,), **kw)
        for k, v in g.items():
            assert (v is not None) == (k in ("dx", "dgate", name)), (name, k)
            assert v is None or torch.equal(v, full[k])
    y, last = ssm.gated_scan_fwd(d["x"], d["gate"], return_last_state=False)
    assert last is None and torch.isfinite(y).all()


def test_on_another_stream():
    """stream=: the call is ordered on that stream, its outputs and workspace belong to it, and inputs may be freed."""
    d = draw(4, 300, 900, "bf16", 1300, rate=True)
    kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}
    y0, l0, c0 = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], **kw)
    g0 = ssm.gated_scan_bwd(d["x"], d["gate"], d["x"], c0, **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for i in range(3):
        side.wait_stream(torch.cuda.current_stream())
        x = d["x"].clone()
        side.wait_stream(torch.cuda.current_stream())
        y, last, ck = ssm.gated_scan_fwd_save(x, d["gate"], h0=d["h0"], stream=side, **kw)
        g = ssm.gated_scan_bwd(x, d["gate"], x, ck, stream=side, **kw)
        del x
        torch.empty_like(y).fill_(float("nan"))  # may not land in x while the side stream reads it
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y0) and torch.equal(last, l0)
        for k in g0:
            assert torch.equal(g[k], g0[k]), k


@pytest.mark.parametrize("L", [40, 1200])
def test_training_step_in_a_graph(L):
    """Forward and backward captured and replayed, new inputs each time, eager work and synchronisations between."""
    d = draw(3, 50, L, "bf16", 1400, rate=True)
    dy = torch.randn_like(d["x"])
    kw = {k: d[k] for k in ("gate_bias", "rate", "z", "reset")}

    def call():
        y, last, ck = ssm.gated_scan_fwd_save(d["x"], d["gate"], h0=d["h0"], mode="convex", **kw)
        return [y, last, *ssm.gated_scan_bwd(d["x"], d["gate"], dy, ck, mode="convex", **kw).values()]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held = call()
    for i in range(3):
        say("gated graph replay %d L=%d" % (i, L))
        d["x"].copy_(torch.randn_like(d["x"]))
        want = [v.clone() for v in call()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(held, want):
            assert torch.equal(u, v)


def test_decode_in_a_graph():
    d = draw(5, 333, 4, "bf16", 1500, rate=True, reset=False)
    x, gate, z = (d[k][..., 0].contiguous() for k in ("x", "gate", "z"))
    state, out = d["h0"].clone(), torch.empty_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        ssm.gated_state_update(state.clone(), x, gate, d["gate_bias"], d["rate"], z, out=out)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ssm.gated_state_update(state, x, gate, d["gate_bias"], d["rate"], z, out=out)
    other = d["h0"].clone()
    state.copy_(d["h0"])
    for t in range(4):
        for dst, k in ((x, "x"), (gate, "gate"), (z, "z")):
            dst.copy_(d[k][..., t])
        want = ssm.gated_state_update(other, x.clone(), gate.clone(), d["gate_bias"], d["rate"], z.clone())
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(state, other)


def test_offsets_past_32_bits():
    """More than 2^31 elements in each stream: the last rows equal the same rows computed alone."""
    batch, dim, L = 1, 1100, 2000003
    say("gated past 2^31 elements: %d x %d" % (dim, L))
    g = torch.Generator(device=DEV).manual_seed(5)
    x = torch.randn((batch, dim, L), generator=g, device=DEV, dtype=torch.bfloat16)
    gate = torch.randn((batch, dim, L), generator=g, device=DEV, dtype=torch.bfloat16)
    assert x.numel() > 2 ** 31
    y, last, ck = ssm.gated_scan_fwd_save(x, gate, mode="convex")
    gr = ssm.gated_scan_bwd(x, gate, x, ck, mode="convex")
    torch.cuda.synchronize()
    for row in (0, dim - 2):
        xs, gs = x[:, row:row + 2].contiguous(), gate[:, row:row + 2].contiguous()
        y1, l1, c1 = ssm.gated_scan_fwd_save(xs, gs, mode="convex")
        g1 = ssm.gated_scan_bwd(xs, gs, xs, c1, mode="convex")
        # the rows alone take more waves each, so sums are grouped differently: a bf16 step at most
        assert torch.allclose(y[:, row:row + 2].float(), y1.float(), rtol=2 ** -7, atol=1e-5)
        assert torch.allclose(last[:, row:row + 2], l1, rtol=1e-4, atol=1e-6)
        assert torch.allclose(ck[:, row:row + 2], c1, rtol=1e-4, atol=1e-5)
        for k in ("dx", "dgate"):
            assert torch.allclose(gr[k][:, row:row + 2].float(), g1[k].float(), rtol=2 ** -7, atol=1e-5), k


def test_refusals_on_the_gpu():
    d = draw(2, 4, 20, "f32", 1600)
    x, gate = d["x"], d["gate"]
    with pytest.raises(ValueError, match="mode"):
        ssm.gated_scan_fwd(x, gate, mode="other")
    with pytest.raises(ValueError, match="contiguous"):
        ssm.gated_scan_fwd(x.transpose(0, 1).contiguous().transpose(0, 1), gate)
    with pytest.raises(ValueError, match="gate"):
        ssm.gated_scan_fwd(x, gate[..., :-1].contiguous())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.gated_scan_fwd(x.half(), gate.half())
    with pytest.raises(TypeError, match="gate"):
        ssm.gated_scan_fwd(x, gate.bfloat16())
    with pytest.raises(TypeError, match="reset"):
        ssm.gated_scan_fwd(x, gate, reset=torch.zeros((2, 20), device=DEV))
    with pytest.raises(ValueError, match="ckpt"):
        ssm.gated_scan_bwd(x, gate, x, torch.zeros((2, 4, 2), device=DEV))
    with pytest.raises(ssm.SsmError, match="SSM_ERR_ALIAS"):
        ssm.gated_scan_fwd(x, gate, out=x)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.gated_scan_fwd(x[..., :0].contiguous(), gate[..., :0].contiguous())
    with pytest.raises(ssm.SsmError, match="SSM_ERR_ALIAS"):
        ssm.gated_state_update(d["h0"], d["h0"], gate[..., 0].contiguous())
