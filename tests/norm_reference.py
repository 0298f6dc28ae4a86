"""Plain float64 form of the norms and their gradients (numpy), with a bound on
each output's fp32 error.

u = 2^-24.  A row's sums are at most 64 additions deep (32 numbers a lane, 6
levels of lanes, 16 waves), so a sum is off by at most 64 u times the sum of
magnitudes; products, the division and the square root add a few u each.  The
column sums run over at most 160 additions in the tests' shapes.
"""
import numpy as np

U = 2.0 ** -24


def forward(x, weight=None, bias=None, residual=None, eps=1e-5, kind="layer", s=None):
    """s: the stored sum (already rounded), by default x + residual as they are."""
    x = np.asarray(x, np.float64)
    if s is None:
        s = x if residual is None else x + np.asarray(residual, np.float64)
    s = np.asarray(s, np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    mean = s.mean(-1) if kind == "layer" else np.zeros(s.shape[:-1])
    c = s - mean[..., None]
    var = (c * c).mean(-1)
    rstd = 1 / np.sqrt(var + eps)
    n = c * rstd[..., None]
    y = n * w + (0.0 if bias is None else np.asarray(bias, np.float64))
    off = 64 * U * np.abs(s).mean(-1) if kind == "layer" else np.zeros_like(mean)  # of the mean
    rel = off * np.abs(c).mean(-1) * rstd ** 2 + 40 * U                             # of rstd, over rstd
    n_err = rstd[..., None] * (off[..., None] + 2 * U * np.abs(s)) + np.abs(n) * (rel[..., None] + 4 * U)
    return dict(y=y, s=s, mean=mean, rstd=rstd, n=n, mean_err=off + U * np.abs(mean), rstd_err=rstd * (rel + 4 * U),
                n_err=n_err, y_err=np.abs(w) * n_err + 2 * U * (np.abs(n * w) + np.abs(y)), rel=rel)


def backward(dy, s, weight=None, dresidual_out=None, eps=1e-5, kind="layer"):
    dy = np.asarray(dy, np.float64)
    f = forward(s, weight, None, None, eps, kind)
    n, n_err, rstd = f["n"], f["n_err"], f["rstd"][..., None]
    w = np.ones(dy.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    g = dy * w
    c2 = (g * n).mean(-1, keepdims=True)
    c2_err = 66 * U * np.abs(g * n).mean(-1, keepdims=True) + (np.abs(g) * n_err).mean(-1, keepdims=True)
    c1 = g.mean(-1, keepdims=True) if kind == "layer" else 0.0
    c1_err = 66 * U * np.abs(g).mean(-1, keepdims=True) if kind == "layer" else 0.0
    inner = g - c1 - n * c2
    ds = rstd * inner
    ds_err = rstd * (3 * U * np.abs(g) + c1_err + 2 * U * np.abs(c1) + n_err * np.abs(c2) + np.abs(n) * c2_err
                     + 3 * U * np.abs(n * c2)) + np.abs(ds) * (f["rel"][..., None] + 4 * U)
    if dresidual_out is not None:
        ds = ds + np.asarray(dresidual_out, np.float64)
        ds_err = ds_err + U * np.abs(ds)
    rows = tuple(range(dy.ndim - 1))
    return dict(dx=ds, dx_err=ds_err, dweight=(dy * n).sum(rows),
                dweight_err=(np.abs(dy) * n_err + 160 * U * np.abs(dy * n)).sum(rows),
                dbias=dy.sum(rows), dbias_err=160 * U * np.abs(dy).sum(rows))
