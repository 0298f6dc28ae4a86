"""Layer and RMS norm (forward, backward) through the C ABI against the float64
form (needs an MI355X).

Every output value is held to its own bound: the fp32 arithmetic's
(norm_reference) plus, for an output in the io or residual type, half a step
of that type (2^-8 relative in bf16, 2^-24 in fp32).
"""
import numpy as np
import pytest
import torch

import norm_reference as ref
import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
TYPES = [(F32, F32), (BF16, BF16), (BF16, F32)]  # io, residual


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def check(got, want, err, what):
    dt, got = got.dtype, np64(got)
    assert got.shape == want.shape, what
    bound = err * (1 + HALF[dt]) + HALF[dt] * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound, at %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / bound), np.argwhere(bad)[0])


def draw(shape, io, res, seed, residual=True, weight=True, bias=True, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    dim = shape[-1]

    def normal(*s):
        return torch.randn(s, generator=g)

    d = dict(x=(normal(*shape) + offset).to(io), residual=(2 * normal(*shape)).to(res) if residual else None,
             weight=1 + 0.3 * normal(dim) if weight else None, bias=0.3 * normal(dim) if bias else None)
    dy, ds = normal(*shape).to(io), normal(*shape).to(res if residual else io)
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}, dy.to(DEV), ds.to(DEV)


def run_all(shape, io, res, kind, seed, what, eps=1e-5, with_ds=True, **opts):
    d, dy, ds = draw(shape, io, res, seed, **opts)
    y, s, mean, rstd = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"], eps=eps, kind=kind)
    g = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds if with_ds else None, kind=kind)
    torch.cuda.synchronize()
    if d["residual"] is None:
        assert s is d["x"]
    else:  # fp32 sum of the two, rounded once to the residual's type
        assert torch.equal(s, (d["x"].float() + d["residual"].float()).to(s.dtype))
    f = ref.forward(np64(d["x"]), np64(d["weight"]), np64(d["bias"]), eps=eps, kind=kind, s=np64(s))
    b = ref.backward(np64(dy), np64(s), np64(d["weight"]), np64(ds) if with_ds else None, eps=eps, kind=kind)
    check(y, f["y"], f["y_err"], what + " y")
    check(rstd, f["rstd"], f["rstd_err"], what + " rstd")
    if kind == "layer":
        check(mean, f["mean"], f["mean_err"], what + " mean")
    else:
        assert mean is None
    check(g["dx"], b["dx"], b["dx_err"], what + " dx")
    if s.dtype != dy.dtype:
        check(g["dresidual"], b["dx"], b["dx_err"], what + " dresidual")
    else:
        assert g["dresidual"] is None
    check(g["dweight"], b["dweight"], b["dweight_err"], what + " dweight")
    check(g["dbias"], b["dbias"], b["dbias_err"], what + " dbias")
    return d, y, s, mean, rstd, g


# Widths on and around 8, 16, 32 and 64 lanes of 8, two and four pieces, two to
# sixteen waves, and the largest; rows that leave groups and blocks part empty.
SHAPES = [(1, 1), (3, 7), (70, 8), (5, 63), (130, 64), (33, 65), (9, 128), (257, 200), (40, 256), (7, 300), (1, 512),
          (21, 513), (5, 768), (66, 1000), (3, 1024), (19, 1025), (2, 2048), (11, 2049), (4, 4096), (3, 5121),
          (2, 8192), (3, 10007), (1, 16384), (2, 16385), (2, 32768), (2500, 96), (1300, 640), (700, 1500), (530, 4100)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_shapes(shape, types):
    io, res = types
    i = SHAPES.index(shape)
    kind = ("layer", "rms")[i % 2]
    say("norm %s io=%s res=%s %s" % (shape, io, res, kind))
    run_all(shape, io, res, kind, i, "%s" % (shape,), residual=i % 3 != 2 or io != res)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [40, 515, 1400, 2900, 5000])
def test_options(dim, types, kind):
    """Each of weight, bias, residual and the gradient past the norm left out."""
    io, res = types
    for k, opts in enumerate([dict(weight=False), dict(bias=False), dict(weight=False, bias=False), dict(with_ds=False),
                              dict(residual=False)]):
        if io != res and not opts.get("residual", True):
            continue
        run_all((2, 9, dim), io, res, kind, 100 + k, "%s" % opts, **opts)


@pytest.mark.parametrize("offset", [10.0, 300.0])
def test_large_mean(offset):
    """Rows whose mean is far above their spread: the variance is summed about the mean, so the bound grows with the
    mean's own rounding only."""
    run_all((50, 1000), F32, F32, "layer", 200, "offset", residual=False, offset=offset)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_constant_and_zero_rows(kind):
    """A constant row has variance 0: y is the bias and rstd 1 / sqrt(eps); a zero row likewise for rms."""
    x = torch.zeros((3, 300), device=DEV)
    x[0] = 5.0
    bias = torch.randn(300, device=DEV)
    y, _, mean, rstd = ssm.norm_fwd(x, bias=bias, kind=kind, eps=1e-5)
    assert torch.equal(y[1:], bias.expand(2, 300))
    assert torch.allclose(rstd[1:], torch.full((2,), 1e-5 ** -0.5, device=DEV), rtol=1e-6)
    if kind == "layer":
        assert torch.equal(y[0], bias) and torch.equal(mean, x[:, 0])


def test_rows_that_are_not_finite_stay_alone():
    for dim in (24, 200, 700, 2900):
        x = torch.randn((9, dim), device=DEV)
        clean = ssm.norm_fwd(x)[0]
        bad = x.clone()
        bad[2, 1], bad[6, dim - 1] = float("inf"), float("nan")
        y = ssm.norm_fwd(bad)[0]
        keep = [0, 1, 3, 4, 5, 7, 8]
        assert torch.equal(y[keep], clean[keep])
        assert torch.isnan(y[2]).any() and torch.isnan(y[6]).all()


def test_residual_in_place():
    for types in TYPES:
        d, _, _ = draw((13, 900), *types, 300)
        want = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])
        r = d["residual"].clone()
        got = ssm.norm_fwd(d["x"], d["weight"], d["bias"], r, residual_out=r)
        assert got[1] is r and torch.equal(r, want[1]) and torch.equal(got[0], want[0])
        y, s, mean, rstd = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"], save_stats=False)
        assert mean is None and rstd is None and torch.equal(y, want[0])


def framed(shape, dtype, offset, fill):
    n = int(np.prod(shape))
    buf = torch.full((n + offset + 64,), fill, dtype=dtype, device=DEV)
    return buf[offset:offset + n].view(shape), buf


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("dim", [5, 64, 333, 1029, 2600])
def test_any_alignment_and_nothing_else_written(dim, types):
    io, res = types
    d, dy, ds = draw((7, dim), io, res, 400)
    y, s, mean, rstd = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])
    g = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds)
    m = {}
    for k, v in dict(d, dy=dy, ds=ds).items():
        m[k], _ = framed(v.shape, v.dtype, 1, 1)
        m[k].copy_(v)
    out, ob = framed((7, dim), io, 1, 9)
    so, sb = framed((7, dim), res, 3, 9)
    y2, s2, mean2, rstd2 = ssm.norm_fwd(m["x"], m["weight"], m["bias"], m["residual"], out=out, residual_out=so)
    g2 = ssm.norm_bwd(m["dy"], s2, rstd2, mean=mean2, weight=m["weight"], dresidual_out=m["ds"])
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(s2, s) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    for b, v, o in ((ob, out, 1), (sb, so, 3)):
        assert (b[:o] == 9).all() and (b[o + v.numel():] == 9).all()
    for k, v in g.items():
        assert v is None or torch.equal(v, g2[k]), k


def test_deterministic_and_need():
    d, dy, ds = draw((3000, 777), BF16, F32, 500)
    y, s, mean, rstd = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])
    a = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds)
    b = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    for need in ((), ("dweight",), ("dbias",)):
        c = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds, need=need)
        for k in ("dweight", "dbias"):
            assert (c[k] is not None) == (k in need)
            assert c[k] is None or torch.equal(c[k], a[k])
        assert torch.equal(c["dx"], a["dx"]) and torch.equal(c["dresidual"], a["dresidual"])


def test_on_another_stream():
    d, dy, ds = draw((2000, 1000), BF16, BF16, 600)
    y0, s0, m0, r0 = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])
    g0 = ssm.norm_bwd(dy, s0, r0, mean=m0, weight=d["weight"], dresidual_out=ds)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        x = d["x"].clone()
        side.wait_stream(torch.cuda.current_stream())
        y, s, m, r = ssm.norm_fwd(x, d["weight"], d["bias"], d["residual"], stream=side)
        g = ssm.norm_bwd(dy, s, r, mean=m, weight=d["weight"], dresidual_out=ds, stream=side)
        del x
        torch.empty_like(y).fill_(float("nan"))
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y0) and torch.equal(s, s0)
        for k in g0:
            assert g0[k] is None or torch.equal(g[k], g0[k]), k


def test_training_step_in_a_graph():
    d, dy, ds = draw((600, 700), BF16, F32, 700)

    def call():
        y, s, mean, rstd = ssm.norm_fwd(d["x"], d["weight"], d["bias"], d["residual"])
        g = ssm.norm_bwd(dy, s, rstd, mean=mean, weight=d["weight"], dresidual_out=ds)
        return [y, s, mean, rstd, *g.values()]

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
        say("norm graph replay %d" % i)
        d["x"].copy_(torch.randn_like(d["x"]))
        want = [v.clone() for v in call()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(held, want):
            assert torch.equal(u, v)


def test_offsets_past_32_bits():
    rows, dim = 1100000, 2000
    say("norm past 2^31 elements: %d x %d" % (rows, dim))
    x = torch.randn((rows, dim), device=DEV, dtype=BF16)
    assert x.numel() > 2 ** 31
    y, _, mean, rstd = ssm.norm_fwd(x)
    g = ssm.norm_bwd(x, x, rstd, mean=mean, need=())
    torch.cuda.synchronize()
    for a in (0, rows - 5):
        xs = x[a:a + 5].contiguous()
        y1, _, m1, r1 = ssm.norm_fwd(xs)
        g1 = ssm.norm_bwd(xs, xs, r1, mean=m1, need=())
        assert torch.equal(y[a:a + 5], y1) and torch.equal(mean[a:a + 5], m1)
        assert torch.equal(g["dx"][a:a + 5], g1["dx"])


def test_refusals_on_the_gpu():
    x = torch.randn((4, 64), device=DEV)
    st = ssm.norm_fwd(x)
    with pytest.raises(ValueError, match="kind"):
        ssm.norm_fwd(x, kind="batch")
    with pytest.raises(ValueError, match="contiguous"):
        ssm.norm_fwd(torch.randn((64, 4), device=DEV).t())
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ssm.norm_fwd(x.half())
    with pytest.raises(TypeError, match="residual"):
        ssm.norm_fwd(x, residual=x.bfloat16())
    with pytest.raises(ValueError, match="residual"):
        ssm.norm_fwd(x, residual_out=torch.empty_like(x))
    with pytest.raises(ValueError, match="mean"):
        ssm.norm_bwd(x, x, st[3])
    with pytest.raises(ssm.SsmError, match="SSM_ERR_ALIAS"):
        ssm.norm_fwd(x, out=x)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.norm_fwd(torch.zeros((0, 64), device=DEV))
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.norm_fwd(torch.zeros((4, 0), device=DEV))
    with pytest.raises(ssm.SsmError, match="SSM_ERR_UNSUPPORTED"):
        ssm.norm_fwd(torch.zeros((1, 32769), device=DEV))
