"""Linear attention (forward, backward, decode step) through the C ABI against
the float64 form (needs an MI355X).

Two kinds of tests hold the values.  Inputs that are small whole numbers with a
decay of 1 have sums that fp32, and bf16 where it rounds, hold exactly: every
output has to be equal to the float64 form's, rounded once.  Other inputs are
held to the bound of linear_attn_reference, value by value.
"""
import pytest
import torch

import linear_attn_reference as ref
import selective_state_space_65_amd as ssm

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F32, BF16 = torch.float32, torch.bfloat16
NAMES = ("q", "k", "v", "rate", "step", "reset", "h0")


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def draw(batch, seqlen, heads, groups, dk, dv, io, seed, step=True, reset=0.0, h0=True, whole=False, rates=(0.002, 0.3)):
    """Inputs on the CPU.  whole: numbers in {-1, 0, 1}, rate 0."""
    g = torch.Generator().manual_seed(seed)

    def values(*s, dtype=io):
        return torch.randint(-1, 2, s, generator=g).to(dtype) if whole else torch.randn(s, generator=g).to(dtype)

    d = dict(q=values(batch, seqlen, groups, dk), k=values(batch, seqlen, groups, dk), v=values(batch, seqlen, heads, dv))
    low, high = rates
    d["rate"] = torch.zeros(heads) if whole else low * (high / low) ** torch.rand(heads, generator=g)
    if step:
        d["step"] = torch.randint(0, 3, (batch, seqlen, heads), generator=g).to(io) if whole else \
            (0.6 * torch.randn((batch, seqlen, heads), generator=g)).exp().to(io)
    if reset:
        d["reset"] = (torch.rand((batch, seqlen), generator=g) < reset).to(torch.uint8)
    if h0:
        d["h0"] = values(batch, heads, dk, dv, dtype=F32)
    dy = values(batch, seqlen, heads, dv)
    dlast = values(batch, heads, dk, dv, dtype=F32)
    return d, dy, dlast


def on_gpu(d):
    return {k: v.to(DEV) for k, v in d.items()}


def same(a, b):
    return torch.allclose(a, b, rtol=0.0, atol=0.0, equal_nan=True)


def run(d, dy=None, dlast=None, scale=1.0):
    t = on_gpu(d)
    y, last, ckpt = ssm.linear_attn_fwd_save(scale=scale, **t)
    out = dict(y=y, last_state=last)
    plain = ssm.linear_attn_fwd(scale=scale, **t)
    assert same(plain[0], y) and same(plain[1], last)
    if dy is not None:
        h0 = t.pop("h0", None)
        g = ssm.linear_attn_bwd(dy=dy.to(DEV), ckpt=ckpt, dlast=None if dlast is None else dlast.to(DEV), scale=scale, **t)
        assert (g["dstep"] is None) == ("step" not in t)
        out.update({k: v for k, v in g.items() if v is not None})
        del h0
    torch.cuda.synchronize()
    return {k: v.cpu() for k, v in out.items()}, ckpt.cpu()


def check(got, want, what):
    for name, x in got.items():
        value, bound = want[name]
        assert x.shape == value.shape, (what, name)
        off = (x.double() - value).abs()
        bad = ~(off <= bound * (1 + 2.0 ** -7) + 1e-37)
        assert not bad.any(), "%s %s: %d of %d off, worst %.3g of its bound, at %s" % (
            what, name, bad.sum(), bad.numel(), (off / bound.clamp(min=1e-300)).max(), bad.nonzero()[0].tolist())


def check_equal(got, want, what):
    for name, x in got.items():
        value = want[name][0].to(x.dtype)
        assert torch.equal(x, value), "%s %s: %d of %d differ, first at %s" % (
            what, name, (x != value).sum(), x.numel(), (x != value).nonzero()[0].tolist())


# Widths on and around 32, 64, 128 and 256 and below 8; lengths on and around a
# chunk (32, 64), a block of 512 and several of them; heads that share q and k.
SHAPES = [(1, 1, 1, 1, 1, 1), (2, 3, 2, 1, 7, 9), (1, 31, 2, 2, 8, 8), (2, 64, 3, 3, 16, 64), (1, 65, 4, 2, 33, 65),
          (3, 127, 5, 1, 64, 128), (1, 200, 2, 2, 128, 32), (2, 250, 2, 1, 100, 130), (1, 130, 3, 3, 129, 200),
          (1, 256, 2, 2, 256, 256), (2, 90, 1, 1, 200, 5)]
LONG = [(1, 513, 3, 1, 32, 40), (2, 1025, 2, 2, 20, 70), (1, 1600, 1, 1, 130, 64), (3, 2050, 2, 1, 8, 136)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_exact(shape, io):
    """Sums of at most 256 products of -1, 0 and 1: exact in bf16 as in fp32, but for the output's own rounding."""
    i = SHAPES.index(shape)
    say("linear attention exact %s %s" % (shape, io))
    d, dy, dlast = draw(*shape, io, i, step=i % 2 == 0, reset=0.04 * (i % 3), h0=i % 4 != 1, whole=True)
    if shape[4] > 128 or shape[5] > 128:  # scores up to 256 in bf16: keep q and dy sparse
        d["q"][..., ::2] = 0
        dy[..., ::2] = 0
    got, _ = run(d, dy, dlast if i % 4 != 1 else None)
    check_equal(got, ref.everything(d, dy, dlast if i % 4 != 1 else None, io=io), str(shape))


@pytest.mark.parametrize("shape", LONG)
def test_exact_long(shape):
    """fp32, over several segments: sums below 2^24 are exact."""
    i = LONG.index(shape)
    say("linear attention exact long %s" % (shape,))
    d, dy, dlast = draw(*shape, F32, 50 + i, step=True, reset=0.003 * (i % 2), whole=True)
    got, _ = run(d, dy, dlast)
    check_equal(got, ref.everything(d, dy, dlast), str(shape))


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES + LONG)
def test_values(shape, io):
    i = (SHAPES + LONG).index(shape)
    say("linear attention %s %s" % (shape, io))
    d, dy, dlast = draw(*shape, io, 100 + i, step=i % 3 != 0, reset=0.01 * (i % 2), h0=i % 4 != 1)
    dlast = dlast if i % 4 != 1 else None
    got, _ = run(d, dy, dlast, scale=0.25)
    check(got, ref.everything(d, dy, dlast, scale=0.25, io=io), str(shape))


# Heads that share q and k, in launches of two roles: two tiles of columns in the main pass, the states' pass alone, the
# main pass alone; and a backward whose passes for q and k have segments of 512 tokens, the last one cut short, where
# that for v has 128.
SHARED = [(7, 300, 6, 3, 40, 136), (2, 1100, 4, 2, 130, 24), (2, 1000, 6, 2, 24, 72), (8, 700, 8, 4, 8, 136)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", SHARED)
def test_shared_heads(shape, io):
    i = SHARED.index(shape)
    say("linear attention shared heads %s %s" % (shape, io))
    d, dy, dlast = draw(*shape, io, 150 + i, reset=0.004)
    got, _ = run(d, dy, dlast, scale=0.25)
    check(got, ref.everything(d, dy, dlast, scale=0.25, io=io), str(shape))
    if io == F32:
        d, dy, dlast = draw(*shape, io, 160 + i, reset=0.004, whole=True)
        got, _ = run(d, dy, dlast)
        check_equal(got, ref.everything(d, dy, dlast), str(shape))


# The rates' gradient is a sum over batch rows and blocks of 512 tokens, by four waves of 64 lanes in strides of 256: two
# waves, three, four, all of them twice, and many blocks of one row.
MANY = [(65, 3, 2, 1, 8, 8), (130, 3, 2, 2, 8, 8), (200, 3, 2, 1, 8, 8), (270, 5, 3, 3, 8, 12), (1, 512 * 70 + 9, 1, 1, 2, 3)]


@pytest.mark.parametrize("io,shape", [(F32, s) for s in MANY] + [(BF16, s) for s in MANY[:4]])
def test_rates_gradient_over_many_blocks(io, shape):
    """Whole numbers: the sum of the double's parts is exact, whatever their order."""
    i = MANY.index(shape)
    say("linear attention many blocks %s %s" % (shape, io))
    d, dy, dlast = draw(*shape, io, 180 + i, reset=0.002, whole=True)
    got, _ = run(d, dy, dlast)
    check_equal(got, ref.everything(d, dy, dlast, io=io), str(shape))


@pytest.mark.parametrize("io", [F32, BF16])
def test_resets_at_every_border(io):
    """Resets on and beside the borders of chunks (32, 64), waves of the decays' kernel (64), blocks (512) and segments, side by
    side, and none: whole numbers (few, so that bf16's sums are exact too), all gradients."""
    d, dy, dlast = draw(3, 1100, 2, 1, 8, 12, io, 21, whole=True)
    d["q"][:, :, :, 2:] = 0
    keep = (torch.arange(1100) % 8 == 0)[None, :, None, None]
    d["v"] = d["v"] * keep
    dy = dy * keep
    d["reset"] = torch.zeros(3, 1100, dtype=torch.uint8)
    d["reset"][0, [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 511, 512, 513, 1023, 1024, 1099]] = 1
    d["reset"][1, 448:576] = 1
    got, _ = run(d, dy, dlast)
    want = ref.everything(d, dy, dlast, io=io)
    check_equal(got, want, "borders")


@pytest.mark.parametrize("shape", [(1, 1, 1, 1, 8, 8), (2, 3, 2, 1, 40, 24), (1, 70, 3, 3, 64, 128), (4, 512, 2, 2, 16, 16)])
def test_few_tokens_round_once(shape):
    """Up to 4096 tokens x heads, bf16 outputs are the fp32 sums (whose parts are exact to 2^-24, within fp32's bound) rounded
    once, half a step: 2^-8 of the value."""
    say("linear attention few tokens %s" % (shape,))
    d, dy, dlast = draw(*shape, BF16, 170, reset=0.01)
    got, _ = run(d, dy, dlast, scale=0.25)
    want = ref.everything(d, dy, dlast, scale=0.25, io=F32)
    check(got, {k: (v, b + 2.0 ** -8 * (v.abs() + b)) for k, (v, b) in want.items()}, str(shape))


@pytest.mark.parametrize("shape", [(2, 700, 8, 4, 64, 128), (4, 2100, 2, 2, 16, 24), (3, 1500, 4, 1, 130, 72)])
@pytest.mark.parametrize("need", [("drate", "dstep", "dh0"), ("dh0",)])
def test_long_calls_round_once(shape, need):
    """However many tokens, and whichever gradients are asked for: bf16 outputs are the fp32 sums rounded once."""
    say("linear attention rounds once %s %s" % (shape, need))
    d, dy, dlast = draw(*shape, BF16, 171, reset=0.01)
    t = on_gpu(d)
    y, last, ckpt = ssm.linear_attn_fwd_save(scale=0.25, **t)
    t.pop("h0")
    g = ssm.linear_attn_bwd(dy=dy.to(DEV), ckpt=ckpt, dlast=dlast.to(DEV), scale=0.25, need=need, **t)
    got = dict(y=y.cpu(), last_state=last.cpu(), **{k: v.cpu() for k, v in g.items() if v is not None})
    want = ref.everything(d, dy, dlast, scale=0.25, io=F32)
    check(got, {k: (v, b + 2.0 ** -8 * (v.abs() + b) if k in got and got[k].dtype == BF16 else b) for k, (v, b) in want.items()},
          str(shape))


@pytest.mark.parametrize("io", [F32, BF16])
def test_checkpoints(io):
    d, _, _ = draw(2, 1100, 2, 2, 24, 40, io, 7)
    got, ckpt = run(d)
    _, _, states = ref.forward(**d)
    size = ref.forward(**dict(d, q=d["q"].abs(), k=d["k"].abs(), v=d["v"].abs(), h0=d["h0"].abs()))[2]
    n = 2 * (1100 + 64) + 160
    assert torch.equal(ckpt[:, :, 0], d["h0"]) and torch.equal(ckpt[:, :, -1], got["last_state"])
    for slot, token in ((1, 512), (2, 1024)):
        assert ((ckpt[:, :, slot].double() - states[token - 1]).abs() <= n * ref.U * size[token - 1]).all()


@pytest.mark.parametrize("io", [F32, BF16])
def test_decays_of_every_size(io):
    """A decay of 1 (step 0), one that is 0 (it drops the state), and small steps behind a large one."""
    d, dy, dlast = draw(2, 300, 3, 3, 40, 24, io, 11)
    d["step"][:, 50:60] = 0
    d["step"][0, 100] = 60000.0
    d["step"][:, 101:140] = 2.0 ** -10
    d["step"][1, 200:210] = 7.0
    d["step"][1, 210, 1] = float("inf")
    d["rate"] = torch.tensor([0.0005, 0.2, 3.0])
    finite = dict(d, step=d["step"].clamp(max=1e9))  # rate x 1e9: a decay of 0 all the same
    got, _ = run(d, dy, dlast)
    want = ref.everything(finite, dy, dlast, io=io)
    for name in ("dstep", "drate"):  # the gradient at an infinite step: 0, as the decay is
        assert not got[name].isnan().any()
    check(got, want, "decays")


@pytest.mark.parametrize("seqlen", [30, 200])
@pytest.mark.parametrize("total", [5.0, 40.0, 80.0])
@pytest.mark.parametrize("constant", [False, True])
def test_decays_keep_their_bits(seqlen, total, constant):
    """One token's value read by all later ones, a decay of e^-total in all: every factor is within a few u = 2^-24 of
    itself, however large its exponent.  A factor's exponent, in whole and rest, is off by u / 2 (1.4 of which 2^x takes over as
    0.35 u), the exponential by 2 u, and a product takes u / 2: below 8 u for the two factors and the products of an output,
    and 4 u more for each chunk of 32 tokens that the state was carried over."""
    k = torch.zeros(1, seqlen, 1, 1)
    k[0, 0] = 1
    one = torch.ones(1, seqlen, 1, 1)
    rate = torch.tensor([total / seqlen])
    step = torch.rand((1, seqlen, 1), generator=torch.Generator().manual_seed(3)) * 2
    step[0, 0] = 0
    steps = torch.ones(seqlen).double().cumsum(0) - 1 if constant else step.double().cumsum(1).flatten()
    want = torch.exp(-rate.double() * steps)
    given = {} if constant else dict(step=step.to(DEV))
    y, last = ssm.linear_attn_fwd(one.to(DEV), k.to(DEV), one.to(DEV), rate.to(DEV), **given)
    bound = (8 + 4 * (torch.arange(seqlen) // 32)) * ref.U
    off = (y.cpu().double().flatten() / want - 1).abs()
    assert (off <= bound).all(), (off / bound).max()
    assert (last.cpu().double().flatten() / want[-1] - 1).abs() <= bound[-1]
    state = torch.ones(1, 1, 1, 1, device=DEV)
    zero = torch.zeros(1, 1, 1, device=DEV)
    ssm.linear_attn_state_update(state, zero, zero, zero, torch.tensor([total], device=DEV))
    assert abs(state.item() / torch.exp(torch.tensor(-total).double()).item() - 1) <= 4 * ref.U


@pytest.mark.parametrize("io", [F32, BF16])
def test_no_gradient_where_the_decay_is_0(io):
    """Decays below the smallest normal float, 2^-126 = e^-87.34, drop the state: their gradient is 0, not what the sums
    that cancel leave over."""
    d, dy, dlast = draw(2, 700, 3, 3, 40, 24, io, 12)
    d["rate"] = torch.ones(3)
    d["step"] = (d["step"].float() * 0.05).to(io)
    for i, s in enumerate((88.0, 92.0, 100.0, 103.5, 104.0)):
        d["step"][:, 100 + 100 * i] = s
    got, _ = run(d, dy, dlast)
    for i in range(5):
        assert (got["dstep"][:, 100 + 100 * i] == 0).all(), i
    check(got, ref.everything(d, dy, dlast, io=io), "dropped")


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("field", ["q", "k", "v", "step"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_not_a_number_stays_behind(io, field, value):
    """A token's NaN or infinity reaches no earlier token, no other head or batch row, and none behind a reset."""
    d, dy, _ = draw(2, 200, 2, 2, 40, 70, io, 13, rates=(0.01, 0.05))
    d["reset"] = torch.zeros(2, 200, dtype=torch.uint8)
    d["reset"][0, 90] = 1
    clean = {k: v.clone() for k, v in d.items()}
    if field == "step":
        if value == float("inf"):
            return  # a decay of 0: test_decays_of_every_size
        d["step"][0, 77, 1] = value
    else:
        d[field][0, 77, 1, 3] = value
    got, _ = run(d, dy)
    want, bad = ref.everything(clean, dy, io=io), ref.everything(d, dy, io=io)
    touched = torch.zeros(2, 200, 2, dtype=torch.bool)  # tokens of the reset's packed sequence, of that head
    touched[0, :90, 1] = True
    for name in ("y", "dq", "dk", "dv"):
        x, (value_, bound) = got[name].double(), want[name]
        keep = ~touched
        assert ((x - value_).abs() <= bound * (1 + 2.0 ** -7) + 1e-37)[keep].all(), name
        if name in ("y", "dq"):  # causal outputs: nothing before the token
            assert ((x - value_).abs() <= bound * (1 + 2.0 ** -7) + 1e-37)[0, :77].all(), name
        fine = bad[name][0].isfinite()  # what the recurrence keeps finite stays so
        assert (x.isfinite() == fine).all(), name
    assert ((got["last_state"].double() - want["last_state"][0]).abs() <= want["last_state"][1] + 1e-37).all()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("field,value", [(f, v) for f in ("q", "k", "v", "step", "dy") for v in (float("nan"), float("inf"))
                                         if (f, v) != ("step", float("inf"))])  # a decay of 0: as above
def test_not_a_number_in_the_steps_gradient(io, field, value):
    """dstep is not finite where the recurrence makes it so: in the same packed sequence and head, on the side of the token
    that its state (k, v), its reads (q, dy) or both (step) reach.  The others keep their value, and resets 0."""
    d, dy, _ = draw(2, 600, 2, 2, 40, 70, io, 14, rates=(0.01, 0.05))
    d["reset"] = torch.zeros(2, 600, dtype=torch.uint8)
    d["reset"][0, [30, 90, 512]] = 1
    clean, clean_dy = {k: v.clone() for k, v in d.items()}, dy.clone()
    where = (0, 77, 1) if field == "step" else (0, 77, 1, 3)
    (dy if field == "dy" else d[field])[where] = value
    got, _ = run(d, dy)
    want, bound = ref.everything(clean, clean_dy, io=io)["dstep"]
    bad = ref.everything(d, dy, io=io)["dstep"][0]
    bad[0, [30, 90, 512]] = want[0, [30, 90, 512]] = 0
    assert not bad.isfinite().all() and (bad == want)[0, 90:].all()
    x = got["dstep"].double()
    assert (x.isfinite() == bad.isfinite()).all()
    # The sums may come from either side: held to what the bound is over a whole block.
    bound = torch.cat([bound[:, :512].amax(1, keepdim=True).expand(-1, 512, -1),
                       bound[:, 512:].amax(1, keepdim=True).expand(-1, 88, -1)], 1)
    assert ((x - want).abs() <= bound)[bad == want].all(), ((x - want).abs() / bound)[bad == want].max()
    assert (x[0, [30, 90, 512]] == 0).all()


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(32, 64), (64, 64), (64, 128), (128, 64), (128, 128), (256, 64)])
@pytest.mark.parametrize("field", ["q", "k", "v", "dy"])
def test_not_a_number_where_tiles_are_fetched_ahead(io, dk, dv, field):
    """Rows of whole 16-byte units, which go straight to LDS a chunk ahead: a chunk that is done again token by token writes over
    what was fetched for the next one.  Values, and what is finite, in front of the token, behind it and behind the reset."""
    d, dy, dlast = draw(1, 330, 2, 2, dk, dv, io, 15, rates=(0.01, 0.05))
    say("linear attention NaN %s %d x %d %s" % (field, dk, dv, io))
    d["reset"] = torch.zeros(1, 330, dtype=torch.uint8)
    d["reset"][0, 201] = 1
    clean, clean_dy = {k: v.clone() for k, v in d.items()}, dy.clone()
    (dy if field == "dy" else d[field])[0, 140, 1, 3] = float("nan")
    got, _ = run(d, dy, dlast)
    want, bad = ref.everything(clean, clean_dy, dlast, io=io), ref.everything(d, dy, dlast, io=io)
    for name in ("y", "last_state", "dq", "dk", "dv", "dh0"):
        x, (value, bound), poisoned = got[name].double(), want[name], bad[name][0]
        assert (x.isfinite() == poisoned.isfinite()).all(), name
        same_ = poisoned == value
        assert ((x - value).abs() <= bound * (1 + 2.0 ** -7) + 1e-37)[same_].all(), name


def test_state_that_is_not_finite_is_dropped():
    d, dy, _ = draw(1, 150, 2, 1, 20, 30, BF16, 17)
    d["h0"][0, 0, 3] = float("inf")
    d["h0"][0, 1, :, 5] = float("nan")
    d["reset"] = torch.zeros(1, 150, dtype=torch.uint8)
    d["reset"][0, 70] = 1
    got, _ = run(d)
    fine = ref.everything(dict(d, h0=torch.zeros_like(d["h0"])), io=BF16)
    assert ((got["y"].double() - fine["y"][0]).abs() <= fine["y"][1] * 1.01 + 1e-37)[:, 70:].all()
    assert ((got["last_state"].double() - fine["last_state"][0]).abs() <= fine["last_state"][1] + 1e-37).all()
    assert not got["y"][0, :70, 0].isfinite().any()
    assert got["y"][0, :70, 1, 5].isnan().all() and got["y"][0, :70, 1, :5].isfinite().all()


@pytest.mark.parametrize("io", [F32, BF16])
def test_prompt_in_parts_then_tokens(io):
    """The state carried from call to call in place; single tokens equal a prompt of one."""
    d, _, _ = draw(2, 150, 4, 2, 48, 36, io, 19)
    want = ref.everything(d, scale=0.5, io=io)
    t = on_gpu(d)
    state = t["h0"].clone()
    ys = []
    for a, b in ((0, 70), (70, 71), (71, 140)):
        part = {k: t[k][:, a:b].contiguous() for k in ("q", "k", "v", "step")}
        y, last = ssm.linear_attn_fwd(rate=t["rate"], h0=state, last_state=state, scale=0.5, **part)
        assert last is state
        ys.append(y)
    one = {k: t[k][:, 140].contiguous() for k in ("q", "k", "v", "step")}
    y1, last1 = ssm.linear_attn_fwd(rate=t["rate"], h0=state, scale=0.5, **{k: v[:, None].contiguous() for k, v in one.items()})
    for i in range(140, 150):
        now = {k: t[k][:, i].contiguous() for k in ("q", "k", "v", "step")}
        y = ssm.linear_attn_state_update(state, now["q"], now["k"], now["v"], t["rate"], step=now["step"], scale=0.5)
        if i == 140:
            assert (state - last1).abs().max() <= 4 * ref.U * last1.abs().max()
        ys.append(y[:, None])
    check(dict(y=torch.cat(ys, 1).cpu(), last_state=state.cpu()), want, "parts")
    del y1


STEPS = [(1, 1, 1, 1, 1), (3, 4, 2, 5, 6), (2, 20, 4, 64, 128), (5, 3, 3, 256, 256), (70, 16, 16, 32, 64), (2, 2, 1, 100, 130),
         (1, 3, 3, 255, 36), (40, 40, 8, 16, 20)]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", STEPS)
def test_state_update(shape, io):
    batch, heads, groups, dk, dv = shape
    i = STEPS.index(shape)
    say("linear attention step %s %s" % (shape, io))
    d, _, _ = draw(batch, 1, heads, groups, dk, dv, io, 200 + i, step=i % 2 == 0)
    want = ref.everything(d, scale=0.3, io=io)
    t = on_gpu(d)
    state = t["h0"]
    out = torch.empty(batch, heads, dv, dtype=io, device=DEV)
    y = ssm.linear_attn_state_update(state, t["q"][:, 0], t["k"][:, 0], t["v"][:, 0], t["rate"],
                                     step=t["step"][:, 0] if "step" in t else None, scale=0.3, out=out)
    assert y is out
    value, bound = want["y"]
    check(dict(y=y.cpu()[:, None], last_state=state.cpu()), want, "step %s" % (shape,))


def test_needless_outputs_are_left_out():
    d, dy, dlast = draw(2, 700, 2, 1, 16, 24, F32, 23)
    t = on_gpu(d)
    h0 = t.pop("h0")
    _, last, ckpt = ssm.linear_attn_fwd_save(h0=h0, **t)
    full = ssm.linear_attn_bwd(dy=dy.to(DEV), ckpt=ckpt, dlast=dlast.to(DEV), **t)
    for need in ((), ("drate",), ("dstep",), ("dh0",)):
        g = ssm.linear_attn_bwd(dy=dy.to(DEV), ckpt=ckpt, dlast=dlast.to(DEV), need=need, **t)
        for k, v in g.items():
            if k in ("drate", "dstep", "dh0") and k not in need:
                assert v is None
            else:
                assert torch.equal(v, full[k]), k
    assert ssm.linear_attn_fwd(h0=h0, return_last_state=False, **t)[1] is None


def test_bool_resets_and_given_outputs():
    d, _, _ = draw(2, 100, 2, 2, 16, 24, BF16, 29, reset=0.1)
    t = on_gpu(d)
    y, last = ssm.linear_attn_fwd(**t)
    out, state = torch.empty_like(y), torch.empty_like(last)
    y2, last2 = ssm.linear_attn_fwd(out=out, last_state=state, **dict(t, reset=t["reset"].bool()))
    assert y2 is out and last2 is state and torch.equal(y, y2) and torch.equal(last, last2)


def test_repeats_are_equal():
    d, dy, dlast = draw(1, 3000, 5, 1, 64, 96, BF16, 31, reset=0.002)
    first, _ = run(d, dy, dlast)
    for _ in range(3):
        again, _ = run(d, dy, dlast)
        assert all(torch.equal(first[k], again[k]) for k in first)


def shifted(t, by):
    """t at an address `by` elements behind a 256-byte boundary, and the buffer around it, 0.5 elsewhere."""
    whole = torch.full((t.numel() + by + 64,), 0.5, dtype=t.dtype, device=DEV)
    view = whole[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view, whole


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 150, 2, 1, 64, 128), (1, 700, 3, 3, 40, 72)])
def test_addresses_that_are_only_element_aligned(io, shape):
    """Other loads than those of 16-byte rows, the same sums: the results are the same bits, and nothing else is written."""
    d, dy, dlast = draw(*shape, io, 61, reset=0.02)
    say("linear attention misaligned %s %s" % (shape, io))
    want, ckpt = run(d, dy, dlast)
    t = {k: shifted(v, i + 1)[0] if v.dtype == io else v.to(DEV) for i, (k, v) in enumerate(d.items())}
    assert any(t[k].data_ptr() % 16 for k in ("q", "k", "v"))
    out, around = shifted(torch.zeros(dy.shape, dtype=io), 3)
    state, beside = shifted(torch.zeros(dlast.shape), 5)
    y, last = ssm.linear_attn_fwd(out=out, last_state=state, **t)
    assert y is out and last is state
    assert torch.equal(y.cpu(), want["y"]) and torch.equal(last.cpu(), want["last_state"])
    for whole, by, n in ((around, 3, y.numel()), (beside, 5, last.numel())):
        assert (whole[:by] == 0.5).all() and (whole[by + n:] == 0.5).all()
    t.pop("h0")
    g = ssm.linear_attn_bwd(dy=shifted(dy, 1)[0], ckpt=shifted(ckpt, 1)[0], dlast=shifted(dlast, 1)[0], **t)
    for k, v in g.items():
        assert torch.equal(v.cpu(), want[k]), k


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("shape", [(3, 4, 2, 8, 12), (2, 3, 1, 33, 130)])
def test_state_update_at_element_aligned_addresses(io, shape):
    batch, heads, groups, dk, dv = shape
    d, _, _ = draw(batch, 1, heads, groups, dk, dv, io, 67)
    t = on_gpu(d)
    rows = [t[k][:, 0].contiguous() for k in ("q", "k", "v", "step")]
    want = t["h0"].clone()
    y = ssm.linear_attn_state_update(want, *rows[:3], t["rate"], step=rows[3])
    state, beside = shifted(t["h0"], 1)
    out, around = shifted(torch.zeros_like(y), 5)
    odd = [shifted(r, i + 1)[0] for i, r in enumerate(rows)]
    ssm.linear_attn_state_update(state, *odd[:3], t["rate"], step=odd[3], out=out)
    assert torch.equal(out, y) and torch.equal(state, want)
    for whole, by, n in ((around, 5, y.numel()), (beside, 1, state.numel())):
        assert (whole[:by] == 0.5).all() and (whole[by + n:] == 0.5).all()


def test_streams():
    """On a side stream, and on two at once: each has a workspace of its own."""
    jobs = [draw(1, 2100, 2, 2, 40, 72, BF16, 37 + i) for i in range(2)]
    want = [run(*j) for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    gpu = [(on_gpu(d), dy.to(DEV), dlast.to(DEV)) for d, dy, dlast in jobs]
    torch.cuda.synchronize()
    got = []
    for (t, dy, dlast), s in zip(gpu, streams):
        t = dict(t)
        h0 = t.pop("h0")
        y, last, ckpt = ssm.linear_attn_fwd_save(h0=h0, stream=s, **t)
        got.append((y, last, ssm.linear_attn_bwd(dy=dy, ckpt=ckpt, dlast=dlast, stream=s, **t)))
    torch.cuda.synchronize()
    for (y, last, g), (w, _) in zip(got, want):
        assert torch.equal(y.cpu(), w["y"]) and torch.equal(last.cpu(), w["last_state"])
        assert all(torch.equal(g[k].cpu(), w[k]) for k in g)


def test_graphs():
    """Two captured training steps on one memory pool, replayed in turn with eager calls between, and a captured decode step."""
    jobs = [draw(1, 1300, 2, 1, 40, 72, BF16, 41 + i) for i in range(2)]
    gpu = [(on_gpu(d), dy.to(DEV), dlast.to(DEV)) for d, dy, dlast in jobs]

    def step(t, dy, dlast):
        t = dict(t)
        h0 = t.pop("h0")
        y, last, ckpt = ssm.linear_attn_fwd_save(h0=h0, **t)
        return dict(y=y, last=last, **ssm.linear_attn_bwd(dy=dy, ckpt=ckpt, dlast=dlast, **t))

    eager = [{k: v.clone() for k, v in step(*j).items()} for j in gpu]
    torch.cuda.synchronize()
    graphs, outs, pool = [], [], None
    for j in gpu:
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
            step(*gpu[turn % 2])
    t = gpu[0][0]
    state, now = t["h0"].clone(), {k: t[k][:, 5].contiguous() for k in ("q", "k", "v", "step")}
    want = state.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = ssm.linear_attn_state_update(state, now["q"], now["k"], now["v"], t["rate"], step=now["step"])
    for _ in range(3):
        g.replay()
        w = ssm.linear_attn_state_update(want, now["q"], now["k"], now["v"], t["rate"], step=now["step"])
        torch.cuda.synchronize()
        assert torch.equal(y, w) and torch.equal(state, want)


def test_offsets_past_32_bits():
    """v and y of more than 2^31 elements: the last tokens, behind a reset, against the float64 form of those alone."""
    heads, dv, seqlen, tail = 16, 256, 540_000, 300
    say("linear attention, %d elements" % (heads * dv * seqlen))
    g = torch.Generator(device=DEV).manual_seed(5)
    q, k = (torch.randn((1, seqlen, 1, 16), generator=g, device=DEV).to(BF16) for _ in range(2))
    v = torch.randn((1, seqlen, heads, dv), generator=g, device=DEV, dtype=BF16)
    rate = torch.full((heads,), 0.01, device=DEV)
    reset = torch.zeros((1, seqlen), dtype=torch.uint8, device=DEV)
    cut = seqlen - tail
    cut -= cut % 512
    reset[0, cut] = 1
    y, last = ssm.linear_attn_fwd(q, k, v, rate, reset=reset)
    torch.cuda.synchronize()
    tail = {n: t[:, cut:].cpu() for n, t in dict(q=q, k=k, v=v).items()}
    check(dict(y=y[:, cut:].cpu(), last_state=last.cpu()), ref.everything(dict(tail, rate=rate.cpu()), io=BF16), "tail")


def test_refusals():
    q, v = torch.zeros(1, 8, 2, 16, device=DEV), torch.zeros(1, 8, 4, 24, device=DEV)
    r, s = torch.ones(4, device=DEV), torch.zeros(1, 4, 16, 24, device=DEV)
    with pytest.raises(ValueError, match="k: expected shape"):
        ssm.linear_attn_fwd(q, q[:, :4].contiguous(), v, r)
    with pytest.raises(TypeError, match="v: expected"):
        ssm.linear_attn_fwd(q, q, v.bfloat16(), r)
    with pytest.raises(ValueError, match="contiguous"):
        ssm.linear_attn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, v, r)
    with pytest.raises(ValueError, match="v must be contiguous"):
        ssm.linear_attn_fwd(q, q, torch.zeros(1, 8, 4, 48, device=DEV)[..., ::2], r)
    with pytest.raises(TypeError, match="rate"):
        ssm.linear_attn_fwd(q, q, v, r.double())
    with pytest.raises(ValueError, match="step"):
        ssm.linear_attn_fwd(q, q, v, r, step=torch.ones(1, 8, 3, device=DEV))
    with pytest.raises(TypeError, match="reset"):
        ssm.linear_attn_fwd(q, q, v, r, reset=torch.zeros(1, 8, device=DEV))
    with pytest.raises(ValueError, match="h0"):
        ssm.linear_attn_fwd(q, q, v, r, h0=s[0])
    with pytest.raises(TypeError, match="io tensors"):
        ssm.linear_attn_fwd(q.half(), q.half(), v.half(), r)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_UNSUPPORTED"):
        ssm.linear_attn_fwd(torch.zeros(1, 8, 2, 300, device=DEV), torch.zeros(1, 8, 2, 300, device=DEV), v, r)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.linear_attn_fwd(torch.zeros(1, 8, 3, 16, device=DEV), torch.zeros(1, 8, 3, 16, device=DEV), v, r)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_SHAPE"):
        ssm.linear_attn_fwd(q[:, :0], q[:, :0], v[:, :0], r)
    with pytest.raises(ssm.SsmError, match="SSM_ERR_ALIAS"):
        ssm.linear_attn_fwd(q, q, v, r, out=v)
    with pytest.raises(ValueError, match="ckpt"):
        ssm.linear_attn_bwd(q, q, v, r, v, s)
    with pytest.raises(ValueError, match="state"):
        ssm.linear_attn_state_update(s[0], q[:, 0], q[:, 0], v[:, 0], r)
