"""The group norm's entry points on the CPU: the float64 form the GPU tests compare
with (against a worked example, torch and central differences), every refusal
of the C ABI on the host, and the binding's."""
import ctypes
import types

import numpy as np
import pytest
import torch

import group_norm_reference as ref
import selective_state_space_65_amd as ssm
from selective_state_space_65_amd import binding

NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 4, 5, 6, 8, 9


def test_worked_example():
    f = ref.forward(np.array([[1.0, 3.0, 5.0, 5.0]]), 2, weight=np.array([2.0, 1.0, 1.0, 1.0]),
                    bias=np.array([0.0, 1.0, 7.0, 0.0]), eps=0.25)
    assert np.allclose(f["y"], [[-2 / np.sqrt(1.25), 1 + 1 / np.sqrt(1.25), 7.0, 0.0]])
    assert f["mean"].tolist() == [[2.0, 5.0]] and np.allclose(f["rstd"], [[1 / np.sqrt(1.25), 2.0]])


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("gated", [False, True])
def test_gradients(kind, activation, gated):
    r = np.random.default_rng(3)
    x, dy, z = r.standard_normal((3, 2, 5, 6)), r.standard_normal((2, 5, 6)), r.standard_normal((2, 5, 6))
    x = x[0] + 0.5
    w, b = r.standard_normal(6), r.standard_normal(6)
    kw = dict(kind=kind, activation=activation)
    g = ref.backward(dy, x, 3, w, b, z if gated else None, **kw)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, b, z)]
    if kind == "layer":
        p = torch.nn.functional.group_norm(t[0].transpose(1, 2), 3, t[1], t[2], 1e-5).transpose(1, 2)
    else:
        q = t[0].reshape(2, 5, 3, 2)
        p = (q / torch.sqrt((q * q).mean((1, 3), keepdim=True) + 1e-5)).reshape(2, 5, 6) * t[1] + t[2]
    y = torch.nn.functional.silu(p) if activation == "silu" else p
    if gated:
        y = y * torch.nn.functional.silu(t[3])
    assert np.allclose(y.detach().numpy(), ref.forward(x, 3, w, b, z if gated else None, **kw)["y"], rtol=1e-12)
    (y * torch.tensor(dy)).sum().backward()
    for k, v in zip(("dx", "dweight", "dbias", "dz"), t):
        if k != "dz" or gated:
            assert np.allclose(g[k], v.grad.numpy(), rtol=1e-10, atol=1e-12), k

    def loss(x_):
        return (ref.forward(x_, 3, w, b, z if gated else None, **kw)["y"] * dy).sum()

    for i in np.ndindex(x.shape):
        up, dn = x.copy(), x.copy()
        up[i] += 1e-6
        dn[i] -= 1e-6
        assert abs((loss(up) - loss(dn)) / 2e-6 - g["dx"][i]) < 1e-6


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def addr(k):
    return (1 << 40) + k * (1 << 36)


def sizes(**over):
    s = dict(batch=4, length=10, channels=64, groups=8, io=0, kind=0, act=0)
    s.update({k: v for k, v in over.items() if k in s})
    return s.values()


def fwd(lib, nbytes=1 << 30, eps=1e-5, **over):
    a = dict(x=addr(1), z=addr(2), weight=addr(3), bias=addr(4), y=addr(5), mean=addr(6), rstd=addr(7), work=addr(8))
    a.update({k: v for k, v in over.items() if k in a})
    v = list(a.values())
    return lib.ssm_group_norm_fwd(*sizes(**over), *v[:4], eps, *v[4:], nbytes, None)


def bwd(lib, nbytes=1 << 30, **over):
    a = dict(dy=addr(1), x=addr(2), z=addr(3), weight=addr(4), bias=addr(5), mean=addr(6), rstd=addr(7), dx=addr(8),
             dz=addr(9), dweight=addr(10), dbias=addr(11), work=addr(12))
    a.update({k: v for k, v in over.items() if k in a})
    return lib.ssm_group_norm_bwd(*sizes(**over), *a.values(), nbytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_common_refusals(lib, call):
    assert call(lib, io=5) == DTYPE
    for name in ("batch", "length", "channels", "groups"):
        assert call(lib, **{name: 0}) == SHAPE, name
    assert call(lib, groups=7) == SHAPE
    assert call(lib, groups=128) == SHAPE
    assert call(lib, batch=1 << 50, length=1 << 12) == SHAPE
    assert call(lib, channels=65537, groups=1) == UNSUPPORTED
    assert call(lib, batch=1 << 27, length=1, channels=512, groups=1) == UNSUPPORTED   # 2^32 lanes, two rows each
    assert call(lib, kind=2) == UNSUPPORTED
    assert call(lib, act=2) == UNSUPPORTED
    assert call(lib, x=None) == NULL
    assert call(lib, work=None) == NULL
    assert call(lib, work=addr(12) + 2) == ALIGN
    assert call(lib, weight=addr(3) + 2) == ALIGN
    assert call(lib, rstd=addr(7) + 1) == ALIGN
    assert call(lib, io=1, z=addr(20) + 1) == ALIGN
    assert call(lib, nbytes=0) == WORKSPACE


def test_forward_refusals(lib):
    assert fwd(lib, y=None) == NULL
    n = ctypes.c_int64(0)
    assert lib.ssm_group_norm_fwd_workspace_bytes(4, 10, 64, 8, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert fwd(lib, nbytes=n.value - 1) == WORKSPACE
    assert lib.ssm_group_norm_fwd_workspace_bytes(4, 1, 64, 8, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ssm_group_norm_fwd_workspace_bytes(4, 1, 4096, 1, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.ssm_group_norm_fwd_workspace_bytes(4, 1, 64, 9, 0, ctypes.byref(n)) == SHAPE
    assert fwd(lib, y=addr(1)) == ALIAS
    assert fwd(lib, y=addr(2)) == ALIAS
    assert fwd(lib, mean=addr(7)) == ALIAS
    assert fwd(lib, rstd=addr(3)) == ALIAS
    assert fwd(lib, work=addr(5)) == ALIAS


def test_backward_refusals(lib):
    for field in ("dy", "mean", "rstd", "dx"):
        assert bwd(lib, **{field: None}) == NULL, field
    n = ctypes.c_int64(0)
    assert lib.ssm_group_norm_bwd_workspace_bytes(4, 10, 64, 8, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(lib, nbytes=n.value - 1) == WORKSPACE
    assert lib.ssm_group_norm_bwd_workspace_bytes(4, 1, 64, 8, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(lib, length=1, nbytes=n.value - 1) == WORKSPACE
    assert bwd(lib, dx=addr(1)) == ALIAS
    assert bwd(lib, dz=addr(8)) == ALIAS
    assert bwd(lib, dweight=addr(11)) == ALIAS
    assert bwd(lib, dbias=addr(7)) == ALIAS
    assert bwd(lib, work=addr(9)) == ALIAS
    assert lib.ssm_group_norm_bwd_workspace_bytes(4, 1, 64, 8, 7, None) == DTYPE


def test_binding_refuses_host_tensors_and_streams_elsewhere():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssm.group_norm_fwd(x, 2)
    with pytest.raises(ValueError, match="GPU"):
        ssm.group_norm_bwd(x, x, x[:, :2], 2)
    x = types.SimpleNamespace(is_cuda=True, device=torch.device("cuda", 0), get_device=lambda: 0)
    side = types.SimpleNamespace(device=torch.device("cuda", 1))
    with pytest.raises(ValueError, match="stream"):
        ssm.group_norm_fwd(x, 2, stream=side)
    with pytest.raises(ValueError, match="stream"):
        ssm.group_norm_bwd(x, x, x, 2, stream=side)
