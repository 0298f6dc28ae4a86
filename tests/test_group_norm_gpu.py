"""Group norm (forward, backward) through the C ABI against the float64 form
(needs an MI355X).

Every output value is held to its own bound: the fp32 arithmetic's
(group_norm_reference) plus, for an output in bf16, half a step of it.
"""
import numpy as np
import pytest
import torch

import group_norm_reference as ref
import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def np64(t):
    return None if t is None else t.detach().float().cpu().numpy().astype(np.float64)


def check(got, want, err, what):
    dt, got = got.dtype, np64(got)
    assert got.shape == want.shape, what
    bound = err * (1 + HALF[dt]) * (1 + 2.0 ** -7) + HALF[dt] * np.abs(want) + 1e-37
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of its bound, at %s" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / bound), np.argwhere(bad)[0])


def draw(shape, io, seed, weight=True, bias=True, gated=True, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    c = shape[-1]

    def normal(*s):
        return torch.randn(s, generator=g)

    d = dict(x=(normal(*shape) * (0.4 * normal(c)).exp() + normal(c) + offset).to(io),
             weight=1 + 0.3 * normal(c) if weight else None, bias=0.3 * normal(c) if bias else None,
             z=normal(*shape).to(io) if gated else None)
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}, normal(*shape).to(io).to(DEV)


def run_all(shape, groups, io, seed, what, kind="layer", activation="none", eps=1e-5, **opts):
    d, dy = draw(shape, io, seed, **opts)
    kw = dict(weight=d["weight"], bias=d["bias"], z=d["z"], kind=kind, activation=activation)
    y, mean, rstd = ssm.group_norm_fwd(d["x"], groups, eps=eps, **kw)
    g = ssm.group_norm_bwd(dy, d["x"], rstd, groups, mean=mean, **kw)
    bare = ssm.group_norm_fwd(d["x"], groups, eps=eps, save_stats=False, **kw)
    torch.cuda.synchronize()
    assert bare[1] is None and bare[2] is None and torch.equal(bare[0], y)
    n64 = {k: np64(v) for k, v in d.items()}
    kw64 = dict(weight=n64["weight"], bias=n64["bias"], z=n64["z"], kind=kind, activation=activation, eps=eps)
    f = ref.forward(n64["x"], groups, **kw64)
    b = ref.backward(np64(dy), n64["x"], groups, **kw64)
    check(y, f["y"], f["y_err"], what + " y")
    check(rstd, f["rstd"], f["rstd_err"], what + " rstd")
    if kind == "layer":
        check(mean, f["mean"], f["mean_err"], what + " mean")
    else:
        assert mean is None
    for k in ("dx", "dweight", "dbias") + (("dz",) if d["z"] is not None else ()):
        check(g[k], b[k], b[k + "_err"], what + " " + k)
    if d["z"] is None:
        assert g["dz"] is None
    return y, mean, rstd, g


# One position: groups on and around 8, 16, 32 and 64 lanes of 8, two and four
# pieces, and above what a wave holds; batch rows that leave blocks part empty.
ROWS = [((1, 8), 1), ((3, 21), 3), ((70, 64), 8), ((5, 63), 1), ((33, 130), 2), ((257, 512), 4), ((9, 1000), 5), ((700, 96), 2),
        ((7, 1539), 3), ((2, 2048), 2), ((3, 2050), 2), ((11, 4096), 2), ((2, 4104), 1), ((1, 20000), 4), ((1, 16), 16),
        ((4000, 256), 16), ((1300, 40), 1)]
# Maps: several columns of threads, groups that cross them, single positions of a run, odd widths.
MAPS = [((2, 2, 8), 1), ((1, 5, 12), 3), ((3, 33, 64), 8), ((2, 7, 9, 30), 5), ((1, 300, 330), 11), ((4, 100, 7), 1),
        ((2, 1000, 96), 4), ((1, 3, 2056), 2), ((2, 40, 4100), 2), ((1, 4096, 64), 64), ((5, 129, 512), 32), ((1, 9, 6000), 1)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("case", ROWS + MAPS)
def test_shapes(case, io):
    shape, groups = case
    i = (ROWS + MAPS).index(case)
    say("group norm %s groups=%d %s" % (shape, groups, io))
    run_all(shape, groups, io, i, "%s %d" % (shape, groups), kind=("layer", "rms")[i % 2],
            activation=("none", "silu")[i // 2 % 2], gated=i % 3 != 2)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("case", [((40, 96), 3), ((3, 50, 40), 5)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_options(case, io, kind, activation):
    for k, opts in enumerate([dict(), dict(weight=False), dict(bias=False), dict(weight=False, bias=False, gated=False),
                              dict(gated=False)]):
        run_all(*case, io, 100 + k, "%s %s" % (case, opts), kind=kind, activation=activation, **opts)


@pytest.mark.parametrize("offset", [10.0, 300.0])
@pytest.mark.parametrize("case", [((50, 1000), 4), ((2, 700, 48), 4)])
def test_large_mean(case, offset):
    run_all(*case, F32, 200, "offset", gated=False, offset=offset)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("channels", [8, 6, 64])
def test_one_number_far_off(io, channels):
    """A run's first position of 1024 times the others' size does not blur them.

    The kernel's means are of numbers less that first one, of size 1024 = M, and are
    joined in at most 300 steps, each off by u M at most: by e = 300 u M in all.  A
    sum of squares Q over N numbers is then off by 2048 u Q in its own additions and by
    2 e times the square root of N Q at most through the means' differences: rstd by
    1024 u + e / sigma of itself, sigma^2 = Q / N.  Sums of squares about the first
    number would be off by up to 256 u N / 2 = 0.25 of rstd here.
    """
    length = 32768
    x = torch.randn((2, length, channels), generator=torch.Generator().manual_seed(7)).to(io)
    x[:, 0] = 1024.0
    want = x.double().var((1, 2), unbiased=False)
    y, mean, rstd = ssm.group_norm_fwd(x.to(DEV), 1, eps=0.0)
    u = 2.0 ** -24
    off = 1024 * u + 300 * u * 1024 / want.sqrt()
    err = (rstd.cpu().double()[:, 0] * want.sqrt() - 1).abs()
    assert (err <= off).all(), (err, off)
    err = (mean.cpu().double()[:, 0] - x.double().mean((1, 2))).abs()
    assert (err <= 300 * u * 1024).all(), err


@pytest.mark.parametrize("shape,groups", [((30000, 2, 8), 1), ((3, 400000, 520), 1), ((5000, 9, 72), 9)])
def test_sums_over_many_rows_and_runs(shape, groups):
    """Columns of one number: a sum that grows beside it rounds it the same way each time, so an error shows as it would in
    a sum of any numbers at worst.  Within the bound that all sums here are held to, 256 additions deep, however many
    positions and batch rows."""
    u, deep = 2.0 ** -24, ref.DEEP
    x = torch.ones(shape, device=DEV)
    x[..., ::2] = -1
    x[:, ::2] *= -1
    dy = torch.full(shape, 1.0 / 3.0, device=DEV)
    say("group norm, long sums %s" % (shape,))
    y, _, rstd = ssm.group_norm_fwd(x, groups, kind="rms", eps=0.0)
    assert torch.equal(y, x)
    g = ssm.group_norm_bwd(dy, x, rstd, groups, kind="rms")
    third, count = dy[0, 0, 0].double().item(), shape[0] * shape[1]
    assert ((g["dbias"].double() / (third * count) - 1).abs() <= deep * u).all()
    even = x[0, 0].double() * (shape[1] % 2) * shape[0]  # positions of one sign left over
    assert ((g["dweight"].double() - third * even).abs() <= deep * u * third * count).all()


@pytest.mark.parametrize("shape,groups", [((24576, 8192), 8192), ((200000, 64), 4), ((700000, 8), 1)])
def test_sums_over_many_rows_of_one_position(shape, groups):
    """As above, where a lane adds the batch rows of its channels."""
    say("group norm, long sums %s" % (shape,))
    x = torch.ones(shape, device=DEV)
    x[:, ::2] = -1
    dy = torch.full(shape, 1.0 / 3.0, device=DEV)
    y, _, rstd = ssm.group_norm_fwd(x, groups, kind="rms", eps=0.0)
    assert torch.equal(y, x)
    g = ssm.group_norm_bwd(dy, x, rstd, groups, kind="rms")
    whole = dy[0, 0].double() * shape[0]
    assert ((g["dbias"].double() / whole - 1).abs() <= ref.DEEP * ref.U).all()
    assert ((g["dweight"].double() / (x[0].double() * whole) - 1).abs() <= ref.DEEP * ref.U).all()


@pytest.mark.parametrize("shape", [(3, 300), (3, 17, 60)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_constant_and_zero_groups(shape, kind):
    """A constant group has variance 0: y is the bias and rstd 1 / sqrt(eps); a zero group likewise for rms."""
    x = torch.zeros(shape, device=DEV)
    if kind == "layer":
        x += 5.0
    bias = torch.linspace(-1, 1, shape[-1], device=DEV)
    y, mean, rstd = ssm.group_norm_fwd(x, 5, bias=bias, kind=kind, eps=2.0 ** -16)
    assert torch.equal(y, bias.expand(shape)) and torch.equal(rstd, torch.full_like(rstd, 256.0))
    if kind == "layer":
        assert torch.equal(mean, torch.full_like(mean, 5.0))


@pytest.mark.parametrize("shape", [(4, 96), (4, 9, 96)])
def test_not_a_number_stays_in_its_group(shape):
    d, dy = draw(shape, F32, 7)
    clean = ssm.group_norm_fwd(d["x"], 4, z=d["z"])
    gc = ssm.group_norm_bwd(dy, d["x"], clean[2], 4, mean=clean[1], z=d["z"])
    x = d["x"].clone()
    x.view(4, -1, 96)[1, 0, 30] = float("nan")
    y, mean, rstd = ssm.group_norm_fwd(x, 4, z=d["z"])
    g = ssm.group_norm_bwd(dy, x, rstd, 4, mean=mean, z=d["z"])
    bad = torch.zeros(shape, dtype=torch.bool, device=DEV)
    bad.view(4, -1, 96)[1, :, 24:48] = True
    for a, b in ((y, clean[0]), (g["dx"], gc["dx"]), (g["dz"], gc["dz"])):
        assert a[bad].isnan().all() and torch.equal(a[~bad], b[~bad])


def test_needless_outputs_are_left_out():
    for shape in ((30, 64), (3, 20, 64)):
        d, dy = draw(shape, BF16, 9)
        kw = dict(weight=d["weight"], bias=d["bias"], z=d["z"], activation="silu")
        _, mean, rstd = ssm.group_norm_fwd(d["x"], 8, **kw)
        full = ssm.group_norm_bwd(dy, d["x"], rstd, 8, mean=mean, **kw)
        for need in ((), ("dweight",), ("dbias",), ("dz",)):
            g = ssm.group_norm_bwd(dy, d["x"], rstd, 8, mean=mean, need=need, **kw)
            for k, v in g.items():
                if k in ("dweight", "dbias", "dz") and k not in need:
                    assert v is None
                else:
                    assert torch.equal(v, full[k]), k


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", [(5, 96), (3, 33), (2, 70, 64), (2, 40, 30), (3, 9, 6)])
def test_addresses_that_are_only_element_aligned(io, shape):
    """The same loads at other addresses: the results are the same bits, and nothing else is written."""
    gen = torch.Generator().manual_seed(71)
    x, z, dy = (torch.randn(shape, generator=gen).to(io).to(DEV) for _ in range(3))
    weight, bias = (torch.randn(shape[-1:], generator=gen).to(DEV) for _ in range(2))

    def shifted(t, by):
        whole = torch.full((t.numel() + by + 64,), 0.5, dtype=t.dtype, device=DEV)
        view = whole[by:by + t.numel()].view(t.shape)
        view.copy_(t)
        return view, whole

    kw = dict(groups=4 if shape[-1] == 64 else 3, activation="silu")
    y, mean, rstd = ssm.group_norm_fwd(x, weight=weight, bias=bias, z=z, **kw)
    g = ssm.group_norm_bwd(dy, x, rstd, mean=mean, weight=weight, bias=bias, z=z, **kw)
    out, around = shifted(torch.zeros_like(y), 3)
    sx, sz, sdy, sw, sb, sm, sr = (shifted(t, i + 1)[0] for i, t in enumerate((x, z, dy, weight, bias, mean, rstd)))
    y2, mean2, rstd2 = ssm.group_norm_fwd(sx, weight=sw, bias=sb, z=sz, out=out, **kw)
    assert y2 is out and torch.equal(y2, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
    assert (around[:3] == 0.5).all() and (around[3 + y.numel():] == 0.5).all()
    h = ssm.group_norm_bwd(sdy, sx, sr, mean=sm, weight=sw, bias=sb, z=sz, **kw)
    assert all(torch.equal(g[k], h[k]) for k in g)


def test_streams_and_graphs():
    jobs = [draw((3, 700, 48), BF16, 11 + i) for i in range(2)] + [draw((500, 256), BF16, 13)]

    def step(d, dy, stream=None):
        kw = dict(weight=d["weight"], bias=d["bias"], z=d["z"], activation="silu", stream=stream)
        y, mean, rstd = ssm.group_norm_fwd(d["x"], 4, **kw)
        return dict(y=y, **ssm.group_norm_bwd(dy, d["x"], rstd, 4, mean=mean, **kw))

    eager = [step(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    side = [step(*j, stream=s) for j, s in zip(jobs, streams)]
    torch.cuda.synchronize()
    for a, b in zip(side, eager):
        assert all(torch.equal(a[k], b[k]) for k in b)
    graphs, outs, pool = [], [], None
    for j in jobs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=pool):
            outs.append(step(*j))
        pool = g.pool()
        graphs.append(g)
    for turn in range(3):
        for g, out, want in zip(graphs, outs, eager):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(out[k], want[k]) for k in want), turn
            step(*jobs[turn % 3])


def test_offsets_past_32_bits():
    """More than 2^31 numbers: the last batch row equals its own call."""
    say("group norm of 2^31 + 2^20 numbers")
    x = torch.empty((2049, 4096, 256), dtype=BF16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    x.normal_(generator=g)
    y, mean, rstd = ssm.group_norm_fwd(x, 8, activation="silu")
    # the same run lengths in both calls are not promised: the values agree to their roundings
    one, m1, r1 = ssm.group_norm_fwd(x[-1:], 8, activation="silu")
    torch.cuda.synchronize()
    # sums at most DEEP additions deep: mean off by DEEP u mean |x| (|x| < 1 on average), the variance by 2 DEEP u of itself
    # (squares, and the mean's part), rstd by half of that, in each of the two calls
    off = ref.DEEP * 2.0 ** -24
    assert (mean[-1] - m1[0]).abs().max() <= 2 * off and (rstd[-1] / r1[0] - 1).abs().max() <= 2 * off
    a, b = y[-1].float(), one[0].float()
    assert ((a - b).abs() <= 2 * HALF[BF16] * b.abs() * 1.01 + 1e-5).all()
    del x, y
    rows = torch.empty((2 ** 31 // 256 + 5, 256), dtype=BF16, device=DEV)
    rows.normal_(generator=g)
    y, _, _ = ssm.group_norm_fwd(rows, 8, kind="rms", save_stats=False)
    one, _, _ = ssm.group_norm_fwd(rows[-3:].contiguous(), 8, kind="rms", save_stats=False)
    assert torch.equal(y[-3:], one)


def test_refusals():
    x = torch.zeros(4, 6, 16, device=DEV)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.group_norm_fwd(x, 3)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.group_norm_fwd(x[:0], 4)
    with pytest.raises(ValueError, match="kind"):
        ssm.group_norm_fwd(x, 4, kind="batch")
    with pytest.raises(ValueError, match="activation"):
        ssm.group_norm_fwd(x, 4, activation="gelu")
    with pytest.raises(ValueError, match="contiguous"):
        ssm.group_norm_fwd(x.transpose(1, 2), 2)
    with pytest.raises(ValueError, match="weight"):
        ssm.group_norm_fwd(x, 4, weight=torch.ones(4, device=DEV))
    with pytest.raises(TypeError, match="z"):
        ssm.group_norm_fwd(x, 4, z=x.bfloat16())
    with pytest.raises(TypeError, match="io tensors"):
        ssm.group_norm_fwd(x.half(), 4)
    with pytest.raises(ValueError, match="batch"):
        ssm.group_norm_fwd(x[0, 0], 4)
    with pytest.raises(ValueError, match="mean"):
        ssm.group_norm_bwd(x, x, torch.ones(4, 4, device=DEV), 4)
    with pytest.raises(ValueError, match="rstd"):
        ssm.group_norm_bwd(x, x, torch.ones(4, 2, device=DEV), 4, kind="rms")


@pytest.mark.parametrize("io", [F32, BF16])
def test_a_layer(io):
    """Norm, linear attention, group norm per head with the output gate: a training step against float64 autograd of the
    same formulas, and a prompt followed by single tokens against the whole."""
    batch, seqlen, heads, d = 2, 150, 3, 32
    width = heads * d
    g = torch.Generator().manual_seed(21)

    def normal(*s):
        return torch.randn(s, generator=g)

    x, z, dy = (normal(batch, seqlen, width).to(io) for _ in range(3))
    q, k = (normal(batch, seqlen, heads, d).to(io) for _ in range(2))
    rate = torch.tensor([0.3, 0.05, 0.01])
    nw, gw = 1 + 0.2 * normal(width), 1 + 0.2 * normal(width)
    t = {n: v.to(DEV) for n, v in dict(x=x, z=z, dy=dy, q=q, k=k, rate=rate, nw=nw, gw=gw).items()}
    n, s, _, rstd = ssm.norm_fwd(t["x"], weight=t["nw"], kind="rms")
    v = n.view(batch, seqlen, heads, d)
    a, _, ckpt = ssm.linear_attn_fwd_save(t["q"], t["k"], v, t["rate"], scale=0.2)
    rows = a.view(-1, width)
    kw = dict(weight=t["gw"], z=t["z"].view(-1, width), kind="rms")
    y, _, grstd = ssm.group_norm_fwd(rows, heads, **kw)
    gg = ssm.group_norm_bwd(t["dy"].view(-1, width), rows, grstd, heads, **kw)
    ga = ssm.linear_attn_bwd(t["q"], t["k"], v, t["rate"], gg["dx"].view_as(a), ckpt, scale=0.2)
    gn = ssm.norm_bwd(ga["dv"].view(batch, seqlen, width), s, rstd, weight=t["nw"], kind="rms")

    leaves = {n_: v_.double().requires_grad_() for n_, v_ in dict(x=x, z=z, q=q, k=k, rate=rate, nw=nw, gw=gw).items()}
    xx = leaves["x"]
    vv = (xx / torch.sqrt((xx * xx).mean(-1, keepdim=True) + 1e-5) * leaves["nw"]).view(batch, seqlen, heads, d)
    order = torch.arange(seqlen)
    lag = (order[:, None] - order).clamp(min=0).double()
    w = torch.exp(-leaves["rate"][:, None, None] * lag) * (order[:, None] >= order)
    score = torch.einsum("bthk,bshk,hts->bhts", leaves["q"], leaves["k"], w)
    aa = 0.2 * torch.einsum("bhts,bshv->bthv", score, vv)
    nn = aa / torch.sqrt((aa * aa).mean(-1, keepdim=True) + 1e-5)
    yy = nn.reshape(batch, seqlen, width) * leaves["gw"] * torch.nn.functional.silu(leaves["z"])
    (yy * dy.double()).sum().backward()
    # Each stored intermediate (n, a, its gradients) is rounded once: a handful of half steps, in the 2-norm
    most = 8 * HALF[io] if io == BF16 else 1e-5
    for got, want, what in ((y, yy, "y"), (gn["dx"], xx.grad, "dx"), (gg["dz"], leaves["z"].grad, "dz"),
                            (ga["dq"], leaves["q"].grad, "dq"), (ga["dk"], leaves["k"].grad, "dk"),
                            (ga["drate"], leaves["rate"].grad, "drate"), (gn["dweight"], leaves["nw"].grad, "dnorm"),
                            (gg["dweight"], leaves["gw"].grad, "dgroup")):
        want = want.detach().reshape(got.shape)
        off = (got.double().cpu() - want).norm() / want.norm()
        assert off <= most, (what, off.item())

    # decode: the last 10 tokens one by one
    cut = seqlen - 10
    part = [u[:, :cut].contiguous() for u in (t["q"], t["k"], v)]
    _, state = ssm.linear_attn_fwd(*part, t["rate"], scale=0.2)
    for i in range(cut, seqlen):
        one = [u[:, i].contiguous() for u in (t["q"], t["k"], v)]
        ai = ssm.linear_attn_state_update(state, *one, t["rate"], scale=0.2)
        yi, _, _ = ssm.group_norm_fwd(ai.view(batch, width), heads, weight=t["gw"], z=t["z"][:, i].contiguous(), kind="rms",
                                      save_stats=False)
        want = yy.detach()[:, i]
        assert (yi.double().cpu() - want).norm() / want.norm() <= most
