"""The norms' entry points on the CPU: the float64 form the GPU tests compare
with (against a worked example, torch autograd and central differences), every
refusal of the C ABI on the host, and the binding's."""
import ctypes

import numpy as np
import pytest
import torch

import norm_reference as ref
import selective_state_space_65_amd as ssm
from selective_state_space_65_amd import binding

NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 4, 5, 6, 8, 9


def test_worked_example():
    f = ref.forward(np.array([[1.0, 3.0]]), weight=np.array([2.0, 1.0]), bias=np.array([0.0, 1.0]), eps=0.0)
    assert f["y"].tolist() == [[-2.0, 2.0]] and f["mean"].tolist() == [2.0] and f["rstd"].tolist() == [1.0]
    f = ref.forward(np.array([[3.0, 4.0]]), residual=np.array([[0.0, 0.0]]), eps=0.0, kind="rms")
    assert np.allclose(f["y"], np.array([[3.0, 4.0]]) / np.sqrt(12.5), atol=1e-15)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_gradients(kind):
    r = np.random.default_rng(3)
    x, dy, ds = r.standard_normal((3, 4, 7)), r.standard_normal((3, 4, 7)), r.standard_normal((3, 4, 7))
    w, b = r.standard_normal(7), r.standard_normal(7)
    g = ref.backward(dy, x, w, ds, kind=kind)
    t = [torch.tensor(v, requires_grad=True) for v in (x, w, b)]
    c = t[0] - t[0].mean(-1, keepdim=True) if kind == "layer" else t[0]
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + 1e-5) * t[1] + t[2]
    assert np.allclose(y.detach().numpy(), ref.forward(x, w, b, kind=kind)["y"], rtol=1e-13)
    ((y * torch.tensor(dy)).sum() + (t[0] * torch.tensor(ds)).sum()).backward()
    for k, v in zip(("dx", "dweight", "dbias"), t):
        assert np.allclose(g[k], v.grad.numpy(), rtol=1e-11, atol=1e-12), k

    def loss(x_):
        return (ref.forward(x_, w, b, kind=kind)["y"] * dy).sum() + (x_ * ds).sum()

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


def fwd(lib, rows=10, dim=64, io=0, res_io=0, kind=0, eps=1e-5, **over):
    a = dict(x=addr(1), residual=addr(2), weight=addr(3), bias=addr(4), y=addr(5), s=addr(6), mean=addr(7),
             rstd=addr(8))
    a.update(over)
    v = list(a.values())
    return lib.ssm_norm_fwd(rows, dim, io, res_io, kind, *v[:4], eps, *v[4:], None)


def bwd(lib, rows=10, dim=64, io=0, res_io=0, kind=0, nbytes=1 << 20, **over):
    a = dict(dy=addr(1), s=addr(2), weight=addr(3), mean=addr(4), rstd=addr(5), ds_out=addr(6), dx=addr(7),
             dres=addr(8), dweight=addr(9), dbias=addr(10), work=addr(11))
    a.update(over)
    return lib.ssm_norm_bwd(rows, dim, io, res_io, kind, *a.values(), nbytes, None)


@pytest.mark.parametrize("call", [fwd, bwd])
def test_common_refusals(lib, call):
    assert call(lib, io=5) == DTYPE
    assert call(lib, io=0, res_io=1) == DTYPE       # an fp32 io with a bf16 residual
    assert call(lib, res_io=9) == DTYPE
    assert call(lib, rows=0) == SHAPE
    assert call(lib, dim=0) == SHAPE
    assert call(lib, rows=1 << 50, dim=1 << 12) == SHAPE
    assert call(lib, dim=32769) == UNSUPPORTED
    assert call(lib, rows=1 << 31, dim=1) == UNSUPPORTED
    if call is fwd:
        assert call(lib, rows=1 << 26, dim=512) == UNSUPPORTED   # 2^32 lanes
    assert call(lib, kind=2) == UNSUPPORTED
    assert call(lib, weight=addr(3) + 2) == ALIGN
    assert call(lib, rstd=addr(8) + 1) == ALIGN


def test_forward_refusals(lib):
    assert fwd(lib, x=None) == NULL
    assert fwd(lib, y=None) == NULL
    assert fwd(lib, residual=None) == NULL                    # an s without a residual
    assert fwd(lib, io=1, res_io=0, residual=None, s=None) == DTYPE
    assert fwd(lib, io=1, res_io=1, x=addr(1) + 1) == ALIGN
    assert fwd(lib, io=1, res_io=0, residual=addr(2) + 2) == ALIGN
    assert fwd(lib, y=addr(1)) == ALIAS
    assert fwd(lib, s=addr(2) + 4) == ALIAS                   # overlapping the residual but not equal to it
    assert fwd(lib, s=addr(2), y=addr(2)) == ALIAS            # y on s
    assert fwd(lib, s=addr(1)) == ALIAS
    assert fwd(lib, mean=addr(8)) == ALIAS
    assert fwd(lib, rstd=addr(3)) == ALIAS


def test_backward_refusals(lib):
    for field in ("dy", "s", "mean", "rstd", "dx", "work"):
        assert bwd(lib, **{field: None}) == NULL, field
    n = ctypes.c_int64(0)
    assert lib.ssm_norm_bwd_workspace_bytes(10, 64, 0, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert bwd(lib, nbytes=n.value - 1) == WORKSPACE
    assert bwd(lib, nbytes=0) == WORKSPACE
    assert bwd(lib, work=addr(11) + 2) == ALIGN
    assert bwd(lib, work=addr(7)) == ALIAS
    assert bwd(lib, dx=addr(1)) == ALIAS
    assert bwd(lib, dres=addr(7)) == ALIAS
    assert bwd(lib, dweight=addr(10)) == ALIAS
    assert bwd(lib, dbias=addr(5)) == ALIAS
    assert lib.ssm_norm_bwd_workspace_bytes(0, 64, 0, 0, ctypes.byref(n)) == SHAPE
    assert lib.ssm_norm_bwd_workspace_bytes(1, 64, 0, 1, ctypes.byref(n)) == DTYPE
    assert lib.ssm_norm_bwd_workspace_bytes(1, 40000, 0, 0, None) == UNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        ssm.norm_fwd(x)
    with pytest.raises(ValueError, match="GPU"):
        ssm.norm_bwd(x, x, x[:, 0])
