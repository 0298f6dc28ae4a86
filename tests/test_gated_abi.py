"""The gated recurrence's entry points on the CPU: every refusal of the C ABI
happens on the host (fake, never-dereferenced addresses), and the binding
refuses tensors it cannot pass on."""
import ctypes
import os
import re

import pytest
import torch

import selective_state_space_65_amd as ssm
from selective_state_space_65_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, ALIGN, ALIAS, UNSUPPORTED, WORKSPACE = 1, 2, 4, 5, 6, 8, 9


@pytest.fixture(scope="module")
def lib():
    return binding.load_library()


def addr(k):
    return (1 << 40) + k * (1 << 36)


def fwd(lib, batch=2, dim=8, seqlen=300, io=0, mode=0, **over):
    a = dict(x=addr(1), gate=addr(2), gate_bias=addr(3), rate=addr(4), z=addr(5), reset=addr(6), h0=addr(7), y=addr(8),
             last=addr(9), ckpt=addr(10))
    a.update(over)
    return lib.ssm_gated_scan_fwd(batch, dim, seqlen, io, mode, *a.values(), None)


def bwd(lib, batch=9, dim=8, seqlen=200, io=0, mode=0, nbytes=None, **over):
    a = dict(x=addr(1), gate=addr(2), gate_bias=addr(3), rate=addr(4), z=addr(5), reset=addr(6), ckpt=addr(7),
             dy=addr(8), dlast=addr(9), dx=addr(10), dgate=addr(11), dgate_bias=addr(12), drate=addr(13), dz=addr(14),
             dh0=addr(15), work=addr(16))
    a.update(over)
    return lib.ssm_gated_scan_bwd(batch, dim, seqlen, io, mode, *a.values(),
                                  2 * batch * dim * 4 if nbytes is None else nbytes, None)


def step(lib, batch=2, dim=8, io=0, mode=0, **over):
    a = dict(state=addr(1), x=addr(2), gate=addr(3), gate_bias=addr(4), rate=addr(5), z=addr(6), y=addr(7))
    a.update(over)
    return lib.ssm_gated_state_update(batch, dim, io, mode, *a.values(), None)


def test_signatures_have_the_headers_argument_counts():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ssm_scan.h")).read(), flags=re.S)
    seen = 0
    for name, args in re.findall(r"\b(ssm_[a-z_0-9]+)\s*\(([^()]*)\)\s*;", text):
        n = 0 if args.strip() in ("", "void") else args.count(",") + 1
        assert len(binding.SIGNATURES[name][1]) == n, name
        for ctype, arg in zip(binding.SIGNATURES[name][1], args.split(",")):
            wide = "int64_t" in arg and "*" not in arg
            assert (ctype is ctypes.c_int64) == wide, (name, arg)
        seen += 1
    assert seen == len(binding.SIGNATURES)


@pytest.mark.parametrize("call", [fwd, bwd, step])
def test_common_refusals(lib, call):
    assert call(lib, io=7) == DTYPE
    assert call(lib, batch=0) == SHAPE
    assert call(lib, dim=-1) == SHAPE
    assert call(lib, batch=1 << 40, dim=1 << 30) == SHAPE
    assert call(lib, batch=1 << 16, dim=1 << 15) == UNSUPPORTED   # 2^31 channels
    if call is not step:
        assert call(lib, batch=1 << 13, dim=1 << 13, seqlen=300) == UNSUPPORTED   # 2^26 rows of 64 lanes
    assert call(lib, mode=3) == UNSUPPORTED
    assert call(lib, mode=-1) == UNSUPPORTED
    assert call(lib, x=addr(1) + 2) == ALIGN
    assert call(lib, io=1, x=addr(1) + 1) == ALIGN
    assert call(lib, gate_bias=addr(3) + 2) == ALIGN
    assert call(lib, rate=addr(4) + 1) == ALIGN


def test_scan_refusals(lib):
    for field in ("x", "gate", "y"):
        assert fwd(lib, **{field: None}) == NULL
    assert fwd(lib, seqlen=0) == SHAPE
    assert fwd(lib, seqlen=1 << 30) == UNSUPPORTED
    assert fwd(lib, y=addr(1)) == ALIAS
    assert fwd(lib, y=addr(6) + 8) == ALIAS             # on the reset bytes
    assert fwd(lib, last=addr(7) + 8) == ALIAS          # overlapping h0 but not equal to it
    assert fwd(lib, last=addr(8) + 16) == ALIAS         # on y
    assert fwd(lib, ckpt=addr(7)) == ALIAS              # on h0
    assert fwd(lib, ckpt=addr(9)) == ALIAS              # on last_state
    assert fwd(lib, h0=addr(9), y=addr(9)) == ALIAS     # h0 = last_state, but y is on both
    assert fwd(lib, h0=addr(7) + 1) == ALIGN


def test_bwd_refusals(lib):
    for field in ("x", "gate", "ckpt", "dy", "dx", "dgate"):
        assert bwd(lib, **{field: None}) == NULL
    assert bwd(lib, seqlen=0) == SHAPE
    assert bwd(lib, nbytes=2 * 9 * 8 * 4 - 1) == WORKSPACE
    assert bwd(lib, nbytes=0) == WORKSPACE
    assert bwd(lib, work=None) == NULL
    assert bwd(lib, work=addr(16) + 2) == ALIGN
    assert bwd(lib, work=addr(10)) == ALIAS             # on dx
    assert bwd(lib, work=addr(7)) == ALIAS              # on the checkpoints
    assert bwd(lib, dx=addr(8)) == ALIAS                # in place of dy
    assert bwd(lib, dgate=addr(2)) == ALIAS
    assert bwd(lib, dgate_bias=addr(13)) == ALIAS       # on drate
    assert bwd(lib, dz=addr(5)) == ALIAS
    assert bwd(lib, dh0=addr(9)) == ALIAS


def test_step_refusals(lib):
    for field in ("state", "x", "gate", "y"):
        assert step(lib, **{field: None}) == NULL
    assert step(lib, y=addr(1)) == ALIAS
    assert step(lib, state=addr(2)) == ALIAS
    assert step(lib, state=addr(1) + 2) == ALIGN


def test_workspace_bytes(lib):
    n = ctypes.c_int64(-1)
    assert lib.ssm_gated_scan_bwd_workspace_bytes(40, 100, 50, 0, ctypes.byref(n)) == 0 and n.value == 2 * 4000 * 4
    assert lib.ssm_gated_scan_bwd_workspace_bytes(1, 100, 50, 1, ctypes.byref(n)) == 0 and n.value == 0
    # none where one block takes every batch row of a channel (small calls)
    assert lib.ssm_gated_scan_bwd_workspace_bytes(32, 100, 50, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(3, 1000, 777, 1, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(4, 4096, 4096, 1, ctypes.byref(n)) == 0 and n.value == 8 * 4 * 4096
    assert lib.ssm_gated_scan_bwd_workspace_bytes(64, 100, 4096, 1, ctypes.byref(n)) == 0 and n.value == 2 * 6400 * 4
    assert lib.ssm_gated_scan_bwd_workspace_bytes(1, 100, 50, 0, None) == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(0, 100, 50, 0, ctypes.byref(n)) == SHAPE
    assert lib.ssm_gated_scan_bwd_workspace_bytes(1, 100, 50, 9, ctypes.byref(n)) == DTYPE


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 4, 8)
    for call in (lambda: ssm.gated_scan_fwd(x, x), lambda: ssm.gated_scan_fwd_save(x, x),
                 lambda: ssm.gated_scan_bwd(x, x, x, torch.zeros(1, 4, 1)),
                 lambda: ssm.gated_state_update(torch.zeros(1, 4), x[..., 0], x[..., 0])):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_ckpt_shape():
    assert ssm.gated_ckpt_shape(2, 5, 1) == (2, 5, 1)
    assert ssm.gated_ckpt_shape(2, 5, 128) == (2, 5, 1)
    assert ssm.gated_ckpt_shape(2, 5, 129) == (2, 5, 2)
