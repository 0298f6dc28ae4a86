"""Plain float64 form of the group norm and its gradients (numpy), with a bound
on each output's fp32 error.

u = 2^-24.  No sum in the tests is more than 256 additions deep (positions of a
thread, threads, channels of a lane, lanes, runs), so it is off by at most
256 u times the sum of magnitudes.  Over a map (length above 1) a channel's numbers
of a run of positions are taken less the run's first, which is at most that channel's
largest deviation away from its mean (their means and squares are then joined, which
is no worse than the plain sums that the bound is for).  The sigmoid is off by 8 u of itself and, through its
argument, by |p| u s (1 - s) <= u / 4; |silu'| <= 1.1 and |silu''| <= 0.5.
"""
import numpy as np

U = 2.0 ** -24
DEEP = 256


def _sigmoid(x):
    return 1 / (1 + np.exp(-x))


def _silu(x):
    """Value, slope, and bounds of their fp32 errors at an exact x."""
    s = _sigmoid(x)
    return x * s, s * (1 + x * (1 - s)), 12 * U * np.abs(x) * s + U, 24 * U


def forward(x, groups, weight=None, bias=None, z=None, eps=1e-5, kind="layer", activation="none"):
    x = np.asarray(x, np.float64)
    shape = x.shape
    batch, channels = shape[0], shape[-1]
    rows = x.reshape(batch, -1, groups, channels // groups)
    length, d = rows.shape[1], rows.shape[3]
    mean = rows.mean((1, 3)) if kind == "layer" else np.zeros((batch, groups))
    c = rows - mean[:, None, :, None]
    var = (c * c).mean((1, 3))
    rstd = 1 / np.sqrt(var + eps)
    if kind == "rms":
        off = np.zeros_like(mean)
        var_err = DEEP * U * var
    elif length == 1:
        off = DEEP * U * np.abs(rows).mean((1, 3))
        var_err = DEEP * U * var + 2 * off * np.abs(c).mean((1, 3)) + off ** 2
    else:
        cm = rows.mean(1)                                            # a channel's own mean
        far = np.abs(rows - cm[:, None]).max(1)
        about = 2 * (rows - cm[:, None]).__pow__(2).mean(1) + 2 * far ** 2  # mean square about the pivot, at most
        cm_err = DEEP * U * np.sqrt(about) + 2 * U * np.abs(cm)
        off = cm_err.mean(2) + DEEP * U * np.abs(cm - mean[..., None]).mean(2) + 2 * U * np.abs(mean)
        var_err = (2 * DEEP * U * about).mean(2) + (2 * np.abs(cm - mean[..., None]) * (cm_err + off[..., None])
                                                    + DEEP * U * (cm - mean[..., None]) ** 2).mean(2) + off ** 2
    rel = 0.5 * var_err / (var + eps) + 8 * U
    n = c * rstd[:, None, :, None]

    def wide(v):
        return v[:, None, :, None]

    n_err = wide(rstd) * (wide(off) + 2 * U * (np.abs(rows) + np.abs(wide(mean)))) + np.abs(n) * (wide(rel) + 4 * U)
    n, n_err = n.reshape(shape), n_err.reshape(shape)
    w = np.ones(channels) if weight is None else np.asarray(weight, np.float64)
    b = np.zeros(channels) if bias is None else np.asarray(bias, np.float64)
    p = n * w + b
    p_err = np.abs(w) * n_err + 2 * U * (np.abs(n * w) + np.abs(p))
    f, slope, f_err, slope_err = (p, np.ones_like(p), p_err, np.zeros_like(p))
    if activation == "silu":
        f, slope, f_err, slope_err = _silu(p)
        f_err, slope_err = f_err + 1.1 * p_err, slope_err + 0.5 * p_err
    y, y_err = f, f_err
    gate = gate_err = gate_slope = gate_slope_err = None
    if z is not None:
        gate, gate_slope, gate_err, gate_slope_err = _silu(np.asarray(z, np.float64))
        y, y_err = f * gate, f_err * (np.abs(gate) + gate_err) + np.abs(f) * gate_err + U * np.abs(f * gate)
    return dict(y=y, y_err=y_err, mean=mean, mean_err=off + U * np.abs(mean), rstd=rstd, rstd_err=rstd * (rel + 4 * U),
                n=n, n_err=n_err, w=w, f=f, f_err=f_err, slope=slope, slope_err=slope_err, gate=gate, gate_err=gate_err,
                gate_slope=gate_slope, gate_slope_err=gate_slope_err, rel=rel)


def backward(dy, x, groups, weight=None, bias=None, z=None, eps=1e-5, kind="layer", activation="none"):
    k = forward(x, groups, weight, bias, z, eps, kind, activation)
    dy = np.asarray(dy, np.float64)
    shape = dy.shape
    batch, channels = shape[0], shape[-1]
    out = {}
    dp, dp_err = dy, np.zeros_like(dy)
    if z is not None:
        out["dz"] = dy * k["f"] * k["gate_slope"]
        out["dz_err"] = np.abs(dy) * (k["f_err"] * (np.abs(k["gate_slope"]) + k["gate_slope_err"])
                                      + np.abs(k["f"]) * k["gate_slope_err"]) + 3 * U * np.abs(out["dz"])
        dp, dp_err = dy * k["gate"], np.abs(dy) * k["gate_err"] + 2 * U * np.abs(dy * k["gate"])
    dp, dp_err = dp * k["slope"], dp_err * (np.abs(k["slope"]) + k["slope_err"]) + np.abs(dp) * k["slope_err"] \
        + 2 * U * np.abs(dp * k["slope"])
    axes = tuple(range(dy.ndim - 1))
    n, n_err, w = k["n"], k["n_err"], k["w"]
    out["dweight"], out["dbias"] = (dp * n).sum(axes), dp.sum(axes)
    out["dweight_err"] = (np.abs(dp) * n_err + dp_err * (np.abs(n) + n_err) + DEEP * U * np.abs(dp * n)).sum(axes)
    out["dbias_err"] = (dp_err + DEEP * U * np.abs(dp)).sum(axes)

    def rows(v):
        return v.reshape(batch, -1, groups, channels // groups)

    def means(v):
        return v.mean((1, 3), keepdims=True)

    g, g_err = rows(dp * w), rows(dp_err * np.abs(w) + U * np.abs(dp * w))
    n, n_err = rows(n), rows(n_err)
    c2 = means(g * n)
    c2_err = means(g_err * (np.abs(n) + n_err) + np.abs(g) * n_err) + (DEEP + 2) * U * means(np.abs(g * n))
    c1 = means(g) if kind == "layer" else 0.0
    c1_err = means(g_err) + (DEEP + 2) * U * means(np.abs(g)) if kind == "layer" else 0.0
    inner = g - c1 - n * c2
    rstd, rel = k["rstd"][:, None, :, None], k["rel"][:, None, :, None]
    err = g_err + c1_err + n_err * np.abs(c2) + np.abs(n) * c2_err + 3 * U * (np.abs(g) + np.abs(c1) + np.abs(n * c2))
    out["dx"] = (rstd * inner).reshape(shape)
    out["dx_err"] = (rstd * err * (1 + rel) + np.abs(rstd * inner) * (rel + 4 * U)).reshape(shape)
    return out
