"""Linear attention's entry points on the CPU: the float64 form the GPU tests
compare with (against a worked example, torch autograd and central
differences), every refusal of the C ABI on the host, and the binding's."""
import ctypes
import types

import pytest
import torch

import linear_attn_reference as ref
import selective_state_space_65_amd as ssm
from selective_state_space_65_amd import binding

NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 4, 5, 6, 8, 9


def draw(batch=2, seqlen=6, heads=4, groups=2, dk=3, dv=5, seed=0, reset=True):
    g = torch.Generator().manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    d = dict(q=normal(batch, seqlen, groups, dk), k=normal(batch, seqlen, groups, dk), v=normal(batch, seqlen, heads, dv),
             rate=torch.rand(heads, generator=g, dtype=torch.float64) + 0.1, step=normal(batch, seqlen, heads).exp(),
             h0=normal(batch, heads, dk, dv), reset=None)
    if reset:
        d["reset"] = torch.zeros(batch, seqlen, dtype=torch.uint8)
        d["reset"][0, 3] = 1
    return d, normal(batch, seqlen, heads, dv), normal(batch, heads, dk, dv)


def test_worked_example():
    one = torch.ones(1, 3, 1, 1, dtype=torch.float64)
    rate = torch.log(torch.tensor([2.0], dtype=torch.float64))     # a = 1/2
    y, last, _ = ref.forward(one, one, one * torch.tensor([4.0, 2.0, 1.0])[None, :, None, None], rate)
    assert torch.allclose(y.flatten(), torch.tensor([4.0, 4.0, 3.0], dtype=torch.float64)) and abs(last.item() - 3.0) < 1e-12
    reset = torch.tensor([[0, 1, 0]], dtype=torch.uint8)
    y, last, _ = ref.forward(one, one, one, rate, reset=reset, h0=torch.full((1, 1, 1, 1), float("inf")))
    assert y.flatten()[0] == float("inf") and torch.allclose(y.flatten()[1:], torch.tensor([1.0, 1.5], dtype=torch.float64))


@pytest.mark.parametrize("reset", [False, True])
def test_gradients(reset):
    """Against autograd through the sum over pairs, and against central differences."""
    d, dy, dlast = draw(reset=reset)
    t = {k: v.clone().requires_grad_() for k, v in d.items() if v is not None and k != "reset"}
    share = t["v"].shape[2] // t["q"].shape[2]
    g = -t["rate"] * t["step"]
    cum = g.cumsum(1)
    part = torch.zeros(d["v"].shape[:2]) if not reset else d["reset"].cumsum(1)
    order = torch.arange(d["v"].shape[1])
    seen = (order[:, None] >= order) & (part[:, :, None] == part[:, None, :])
    w = torch.where(seen[..., None], torch.exp((cum[:, :, None] - cum[:, None]).clamp(max=0)), torch.zeros(()).double())
    q, k = t["q"].repeat_interleave(share, 2), t["k"].repeat_interleave(share, 2)
    score = torch.einsum("bthk,bshk->btsh", q, k) * w
    carry = torch.where((part == 0)[..., None], torch.exp(cum), torch.zeros(()).double())
    y = 0.5 * (torch.einsum("btsh,bshv->bthv", score, t["v"]) + carry[..., None] * torch.einsum("bthk,bhkv->bthv", q, t["h0"]))
    last = torch.einsum("bsh,bshk,bshv->bhkv", w[:, -1], k, t["v"]) + carry[:, -1, :, None, None] * t["h0"]
    ry, rlast, _ = ref.forward(scale=0.5, **d)
    assert torch.allclose(y, ry, rtol=1e-12) and torch.allclose(last, rlast, rtol=1e-12)
    ((y * dy).sum() + (last * dlast).sum()).backward()
    got = ref.backward(dy=dy, dlast=dlast, scale=0.5, **d)
    for name, of in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("drate", "rate"), ("dstep", "step"), ("dh0", "h0")):
        assert torch.allclose(got[name], t[of].grad, rtol=1e-10, atol=1e-12), name

    def loss(**over):
        y_, last_, _ = ref.forward(scale=0.5, **dict(d, **over))
        return ((y_ * dy).sum() + (last_ * dlast).sum()).item()

    for name, of in (("dk", "k"), ("drate", "rate"), ("dstep", "step")):
        for i in range(d[of].numel()):
            up, dn = d[of].clone(), d[of].clone()
            up.view(-1)[i] += 1e-6
            dn.view(-1)[i] -= 1e-6
            assert abs((loss(**{of: up}) - loss(**{of: dn})) / 2e-6 - got[name].reshape(-1)[i].item()) < 1e-6, name


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def addr(k):
    return (1 << 40) + k * (1 << 36)


def sizes(**over):
    s = dict(batch=2, seqlen=600, heads=4, groups=2, dk=64, dv=64, io=0)
    s.update({k: v for k, v in over.items() if k in s})
    return s


def fwd(lib, nbytes=1 << 34, scale=1.0, **over):
    a = dict(q=addr(1), k=addr(2), v=addr(3), rate=addr(4), step=addr(5), reset=addr(6), h0=addr(7), y=addr(8),
             last=addr(9), ckpt=addr(10), work=addr(11))
    a.update({k: v for k, v in over.items() if k in a})
    v = list(a.values())
    return lib.ssm_linear_attn_fwd(*sizes(**over).values(), *v[:7], scale, *v[7:], nbytes, None)


def bwd(lib, nbytes=1 << 34, scale=1.0, **over):
    a = dict(q=addr(1), k=addr(2), v=addr(3), rate=addr(4), step=addr(5), reset=addr(6), ckpt=addr(7), dy=addr(8),
             dlast=addr(9), dq=addr(10), dkk=addr(11), dvv=addr(12), drate=addr(13), dstep=addr(14), dh0=addr(15),
             work=addr(16))
    a.update({k: v for k, v in over.items() if k in a})
    v = list(a.values())
    return lib.ssm_linear_attn_bwd(*sizes(**over).values(), *v[:7], scale, *v[7:], nbytes, None)


def upd(lib, scale=1.0, **over):
    a = dict(state=addr(1), q=addr(2), k=addr(3), v=addr(4), rate=addr(5), step=addr(6), y=addr(7))
    a.update({k: v for k, v in over.items() if k in a})
    s = sizes(**over)
    del s["seqlen"]
    v = list(a.values())
    return lib.ssm_linear_attn_state_update(*s.values(), *v[:6], scale, *v[6:], None)


@pytest.mark.parametrize("call", [fwd, bwd, upd])
def test_common_refusals(lib, call):
    assert call(lib, io=5) == DTYPE
    for name in ("batch", "heads", "groups", "dk", "dv"):
        assert call(lib, **{name: 0}) == SHAPE, name
    assert call(lib, heads=4, groups=3) == SHAPE
    assert call(lib, heads=2, groups=4) == SHAPE
    assert call(lib, batch=1 << 50, heads=1 << 12, groups=1) == SHAPE
    assert call(lib, dk=257) == UNSUPPORTED
    assert call(lib, dv=257) == UNSUPPORTED
    assert call(lib, heads=16385, groups=1) == UNSUPPORTED
    assert call(lib, batch=1 << 26, heads=4) == UNSUPPORTED
    assert call(lib, q=None) == NULL
    assert call(lib, k=None) == NULL
    assert call(lib, v=None) == NULL
    assert call(lib, rate=None) == NULL
    assert call(lib, rate=addr(30) + 2) == ALIGN
    assert call(lib, q=addr(30) + 2) == ALIGN
    assert call(lib, io=1, step=addr(30) + 1) == ALIGN


def test_batch_rows_times_heads(lib):
    """2^20 and more are refused but for the decode step; one below is only refused for what else is wrong with it."""
    for call in (fwd, bwd):
        few = dict(seqlen=1, heads=4, groups=4, dk=8, dv=8)
        assert call(lib, batch=1 << 18, **few) == UNSUPPORTED
        assert call(lib, batch=(1 << 18) - 1, q=None, **few) == NULL
    assert upd(lib, batch=1 << 18, heads=4, groups=4, dk=8, dv=8, q=None) == NULL


def test_forward_refusals(lib):
    assert fwd(lib, seqlen=0) == SHAPE
    assert fwd(lib, y=None) == NULL
    n = ctypes.c_int64(0)
    assert lib.ssm_linear_attn_fwd_workspace_bytes(1, 4096, 2, 2, 64, 64, 0, ctypes.byref(n)) == 0 and n.value > 0
    few = dict(batch=1, seqlen=4096, heads=2, groups=2)
    assert fwd(lib, nbytes=n.value - 1, **few) == WORKSPACE
    assert fwd(lib, work=None, **few) == NULL
    assert fwd(lib, work=addr(11) + 4, **few) == ALIGN
    assert fwd(lib, work=addr(8), **few) == ALIAS
    assert lib.ssm_linear_attn_fwd_workspace_bytes(1, 64, 2, 2, 64, 64, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert fwd(lib, y=addr(1)) == ALIAS
    assert fwd(lib, last=addr(7) + 4) == ALIAS       # overlapping h0 but not equal to it
    assert fwd(lib, last=addr(8)) == ALIAS
    assert fwd(lib, ckpt=addr(7)) == ALIAS
    assert fwd(lib, ckpt=addr(9)) == ALIAS
    assert fwd(lib, last=addr(7) + 2, h0=addr(7) + 2) == ALIGN
    assert lib.ssm_linear_attn_fwd_workspace_bytes(1, 0, 2, 2, 64, 64, 0, ctypes.byref(n)) == SHAPE
    assert lib.ssm_linear_attn_fwd_workspace_bytes(1, 64, 2, 2, 300, 64, 0, None) == UNSUPPORTED


def test_backward_refusals(lib):
    assert bwd(lib, seqlen=0) == SHAPE
    for field in ("ckpt", "dy", "dq", "dkk", "dvv", "work"):
        assert bwd(lib, **{field: None}) == NULL, field
    n, m = ctypes.c_int64(0), ctypes.c_int64(0)
    s = tuple(sizes().values())
    assert lib.ssm_linear_attn_bwd_workspace_bytes(*s, 1, ctypes.byref(n)) == 0
    assert lib.ssm_linear_attn_bwd_workspace_bytes(*s, 0, ctypes.byref(m)) == 0 and 0 < m.value < n.value
    assert bwd(lib, nbytes=n.value - 1) == WORKSPACE
    assert bwd(lib, nbytes=m.value - 1, drate=None, dstep=None) == WORKSPACE
    assert bwd(lib, work=addr(16) + 4) == ALIGN
    assert bwd(lib, work=addr(10)) == ALIAS
    assert bwd(lib, dq=addr(1)) == ALIAS
    assert bwd(lib, dkk=addr(10)) == ALIAS
    assert bwd(lib, dvv=addr(8)) == ALIAS
    assert bwd(lib, drate=addr(4)) == ALIAS
    assert bwd(lib, dstep=addr(5)) == ALIAS
    assert bwd(lib, dh0=addr(9)) == ALIAS


def test_update_refusals(lib):
    assert upd(lib, state=None) == NULL
    assert upd(lib, y=None) == NULL
    assert upd(lib, state=addr(1) + 2) == ALIGN
    assert upd(lib, state=addr(4)) == ALIAS
    assert upd(lib, y=addr(1)) == ALIAS
    assert upd(lib, y=addr(2)) == ALIAS


def test_binding_refuses_host_tensors():
    q, v, r = torch.zeros(1, 4, 1, 8), torch.zeros(1, 4, 2, 8), torch.zeros(2)
    s = torch.zeros(1, 2, 8, 8)
    for call in (lambda: ssm.linear_attn_fwd(q, q, v, r), lambda: ssm.linear_attn_fwd_save(q, q, v, r),
                 lambda: ssm.linear_attn_bwd(q, q, v, r, v, s), lambda: ssm.linear_attn_state_update(s, q[0], q[0], v[0], r)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_stream_of_another_device_is_refused():
    x = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0), get_device=lambda: 0)
    side = types.SimpleNamespace(device=torch.device("cuda", 1))
    for call in (lambda: ssm.linear_attn_fwd(x, x, x, x, stream=side), lambda: ssm.linear_attn_fwd_save(x, x, x, x, stream=side),
                 lambda: ssm.linear_attn_bwd(x, x, x, x, x, x, stream=side),
                 lambda: ssm.linear_attn_state_update(x, x, x, x, x, stream=side)):
        with pytest.raises(ValueError, match="stream"):
            call()


def test_checkpoint_shape():
    assert ssm.linear_attn_ckpt_shape(2, 1, 3, 4, 5) == (2, 3, 2, 4, 5)
    assert ssm.linear_attn_ckpt_shape(2, 512, 3, 4, 5) == (2, 3, 2, 4, 5)
    assert ssm.linear_attn_ckpt_shape(2, 513, 3, 4, 5) == (2, 3, 3, 4, 5)
