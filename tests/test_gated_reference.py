"""The float64 gated recurrence the GPU tests compare with: a worked example,
its gradients against central differences and torch autograd, and a sequence
cut in two."""
import numpy as np
import pytest
import torch

import gated_reference as ref

MODES = ["plain", "convex", "norm"]


def draw(batch, dim, L, seed, rate=False, z=True, reset=True, h0=True):
    r = np.random.default_rng(seed)
    d = dict(x=r.standard_normal((batch, dim, L)), gate=r.standard_normal((batch, dim, L)),
             gate_bias=r.uniform(0, 3, dim), rate=r.uniform(0.05, 2, dim) if rate else None,
             z=r.standard_normal((batch, dim, L)) if z else None,
             reset=(r.random((batch, L)) < 0.2).astype(np.uint8) if reset else None,
             h0=r.standard_normal((batch, dim)) if h0 else None)
    return d, r


def test_worked_example():
    """Two tokens, gate logits 0 (a = 1/2): h = 1/2 h0 + w x by hand."""
    x = np.array([[[2.0, -1.0]]])
    g = np.zeros((1, 1, 2))
    f = ref.forward(x, g, h0=np.array([[4.0]]), mode="plain")
    assert f["states"].tolist() == [[[4.0, 1.0]]]
    f = ref.forward(x, g, h0=np.array([[4.0]]), mode="convex")
    assert f["states"].tolist() == [[[3.0, 1.0]]]
    f = ref.forward(x, g, h0=np.array([[4.0]]), mode="norm")
    w = np.sqrt(0.75)
    assert np.allclose(f["states"], [[[2 + 2 * w, 1 + w - w]]], atol=1e-15)
    f = ref.forward(x, g, h0=np.array([[4.0]]), reset=np.array([[0, 1]]), mode="plain")
    assert f["states"].tolist() == [[[4.0, -1.0]]]
    f = ref.forward(x, g, rate=np.array([2 * np.log(4.0)]), h0=np.array([[4.0]]), mode="convex")  # a = 1/4
    assert np.allclose(f["states"], [[[2.5, 0.625 - 0.75]]], atol=1e-15)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rate", [False, True])
def test_gradients_against_differences(mode, rate):
    d, r = draw(2, 2, 5, [7, rate], rate=rate)
    dy, dlast = r.standard_normal((2, 2, 5)), r.standard_normal((2, 2))
    g = ref.backward(d["x"], d["gate"], dy, d["gate_bias"], d["rate"], d["z"], d["reset"], d["h0"], dlast, mode)

    def loss(**over):
        f = ref.forward(**{**d, **over}, mode=mode)
        return (f["y"] * dy).sum() + (f["last"] * dlast).sum()

    names = dict(x="dx", gate="dgate", gate_bias="dgate_bias", z="dz", h0="dh0", **({"rate": "drate"} if rate else {}))
    for name, gname in names.items():
        v = d[name]
        for i in np.ndindex(v.shape):
            e = 1e-6
            up, dn = v.copy(), v.copy()
            up[i] += e
            dn[i] -= e
            num = (loss(**{name: up}) - loss(**{name: dn})) / (2 * e)
            assert abs(num - g[gname][i]) <= 1e-7 * (1 + abs(num)), (name, i)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("rate", [False, True])
def test_gradients_against_autograd(mode, rate):
    d, r = draw(2, 3, 9, [8, rate], rate=rate)
    dy, dlast = r.standard_normal((2, 3, 9)), r.standard_normal((2, 3))
    t = {k: torch.tensor(v, requires_grad=True) for k, v in d.items() if v is not None and k != "reset"}
    s = torch.sigmoid(t["gate"] + t["gate_bias"][:, None])
    a = torch.exp(-t["rate"][:, None] * s) if rate else s
    w = {"plain": torch.ones_like(a), "convex": 1 - a, "norm": torch.sqrt(1 - a * a)}[mode]
    keep = a * torch.tensor(d["reset"] == 0)[:, None, :]
    h, hs = t["h0"], []
    for i in range(9):
        h = keep[..., i] * h + w[..., i] * t["x"][..., i]
        hs.append(h)
    y = torch.stack(hs, -1) * torch.nn.functional.silu(t["z"])
    ((y * torch.tensor(dy)).sum() + (h * torch.tensor(dlast)).sum()).backward()
    g = ref.backward(d["x"], d["gate"], dy, d["gate_bias"], d["rate"], d["z"], d["reset"], d["h0"], dlast, mode)
    for k, v in t.items():
        assert np.allclose(g["d" + k], v.grad.numpy(), rtol=1e-10, atol=1e-11), k


def test_cut_in_two():
    d, _ = draw(2, 3, 12, 9)
    whole = ref.forward(**d, mode="norm")
    cut = {k: (v[..., :5] if v is not None and k in ("x", "gate", "z", "reset") else v) for k, v in d.items()}
    rest = {k: (v[..., 5:] if v is not None and k in ("x", "gate", "z", "reset") else v) for k, v in d.items()}
    one = ref.forward(**cut, mode="norm")
    two = ref.forward(**{**rest, "h0": one["last"]}, mode="norm")
    assert np.array_equal(np.concatenate([one["y"], two["y"]], -1), whole["y"])
