"""Layer norm of rows and its gradients in 64 bits (numpy), with bounds on what
a 32-bit evaluation may be off by.

    mean = sum x / n;  rstd = (sum (x - mean)^2 / n + eps)^-1/2
    y = (x - mean) rstd weight + bias           (rms: mean = 0)

Bounds.  A sum of n terms taken by at least eight lanes (n / 8 terms each, then
joined) is off by at most k = (n / 8 + 16) 2^-24 of the sum of the terms'
magnitudes.  The constants below count the roundings of 2^-24 that follow.
"""
import numpy as np

U = 2.0 ** -24


def _k(n):
    return (n / 8 + 16) * U


def statistics(x, eps, rms=False):
    x = np.asarray(x, dtype=np.float64)
    mean = np.zeros(x.shape[0]) if rms else x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def layer_norm(x, weight, bias, eps, rms=False):
    """(y, mean, rstd) and their bounds."""
    x = np.asarray(x, dtype=np.float64)
    n = x.shape[1]
    w = np.ones(n) if weight is None else np.asarray(weight, dtype=np.float64)
    b = np.zeros(n) if bias is None else np.asarray(bias, dtype=np.float64)
    mean, rstd = statistics(x, eps, rms)
    y = (x - mean[:, None]) * rstd[:, None] * w + b
    e_mean = np.zeros_like(mean) if rms else (_k(n) + U) * np.abs(x).mean(axis=1)
    # the squares: each x - mean is off by e_mean + U |x - mean|, relative to their root mean square by
    # e_mean rstd; the sum by k; the root halves it, and rounds
    rel = (e_mean * rstd) ** 2 + 2 * U + _k(n) + 4 * U
    e_rstd = rstd * rel
    c = np.abs(x - mean[:, None])
    e_y = ((e_mean[:, None] + U * c) * rstd[:, None] + c * e_rstd[:, None]) * np.abs(w) \
        + 4 * U * (c * rstd[:, None] * np.abs(w) + np.abs(b))
    return (y, mean, rstd), (e_y, e_mean, e_rstd)


def layer_norm_backward(dy, x, weight, mean, rstd, rms=False):
    """{"dx", "dweight", "dbias"} for the given mean and rstd, and their bounds."""
    dy, x = np.asarray(dy, dtype=np.float64), np.asarray(x, dtype=np.float64)
    rows, n = x.shape
    w = np.ones(n) if weight is None else np.asarray(weight, dtype=np.float64)
    m = np.zeros(rows) if rms else np.asarray(mean, dtype=np.float64)
    r = np.asarray(rstd, dtype=np.float64)
    xh = (x - m[:, None]) * r[:, None]
    d = dy * w
    s1 = np.zeros(rows) if rms else d.mean(axis=1)
    s2 = (d * xh).mean(axis=1)
    dx = r[:, None] * (d - s1[:, None] - xh * s2[:, None])
    k = _k(n) + 4 * U
    e1 = 0.0 if rms else k * np.abs(d).mean(axis=1)
    e2 = k * np.abs(d * xh).mean(axis=1)
    e_dx = r[:, None] * (np.add(e1, np.zeros(rows))[:, None] + np.abs(xh) * e2[:, None]
                         + 6 * U * (np.abs(d) + np.abs(s1)[:, None] + np.abs(xh * s2[:, None])))
    ks = (rows + 8) * U   # rows added one after the other at worst
    return ({"dx": dx, "dweight": (dy * xh).sum(axis=0), "dbias": dy.sum(axis=0)},
            {"dx": e_dx, "dweight": ks * np.abs(dy * xh).sum(axis=0), "dbias": ks * np.abs(dy).sum(axis=0)})
