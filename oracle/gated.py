"""The gated linear recurrence and its gradients in 64 bits (numpy), one token
at a time, with bounds on what a 32-bit evaluation may be off by.

    a = 1/(1+e^-g) or e^g;  w = 1 or 1 - a;  h_t = a_t h_{t-1} + w_t x_t

Arrays are (batch, len, channels); states (batch, channels).

Bounds.  A chunked evaluation forms every product of gates and every sum of
the expanded h_t = sum_s (a_t ... a_{s+1}) w_s x_s in 32 bits, in some order.
Token r's step adds to each of its terms the relative error c_r of its gate
and a few roundings of 2^-24 (product, sum, the joining of chunks).  With
M_t = a_t M_{t-1} + |w_t x_t| the sum of the terms' magnitudes, the error of
h_t is at most E_t = a_t E_{t-1} + c_t M_t.  A gate's relative error is at
most that of its exponential: its argument is rounded (|g| 2^-24 after the
product with log2 e, and once more inside), the function itself is off by
2^-22 and the reciprocal by 2^-23; c = 2^-20 + |g| 2^-22 holds all of it and
the roundings.  1 - a is formed without cancellation and obeys the same c.
"""
import numpy as np


def decay(g, log, convex):
    """a, w and 1 - a."""
    g = np.asarray(g, dtype=np.float64)
    with np.errstate(over="ignore"):
        if log:
            a, one_less = np.exp(g), -np.expm1(g)
        else:
            a, one_less = 1.0 / (1.0 + np.exp(-g)), 1.0 / (1.0 + np.exp(g))
    return a, (one_less if convex else np.ones_like(a)), one_less


def _step_error(g, a):
    return 2.0 ** -20 + np.where(a > 0, np.abs(np.where(np.isfinite(g), g, 0.0)), 0.0) * 2.0 ** -22


def scan(x, g, log=False, convex=False, h0=None):
    """h (batch, len, channels), and the bound E of its 32-bit error."""
    x, g = np.asarray(x, dtype=np.float64), np.asarray(g, dtype=np.float64)
    a, w, _ = decay(g, log, convex)
    c = _step_error(g, a)
    h = np.zeros((x.shape[0], x.shape[2])) if h0 is None else np.asarray(h0, dtype=np.float64).copy()
    big, err = np.abs(h), np.zeros_like(h)
    hs, errs = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1]):
        b = w[:, t] * x[:, t]
        h = a[:, t] * h + b
        big = a[:, t] * big + np.abs(b)
        err = a[:, t] * err + c[:, t] * big
        hs[:, t], errs[:, t] = h, err
    return hs, errs


def scan_backward(x, g, dy, log=False, convex=False, h0=None, dh=None):
    """{"dx", "dgate", "d_initial_state"} and their bounds, as a second dict."""
    x, g, dy = (np.asarray(v, dtype=np.float64) for v in (x, g, dy))
    a, w, one_less = decay(g, log, convex)
    c = _step_error(g, a)
    first = np.zeros((x.shape[0], x.shape[2])) if h0 is None else np.asarray(h0, dtype=np.float64)
    hs, errs = scan(x, g, log, convex, h0)
    before = np.concatenate((first[:, None], hs[:, :-1]), axis=1)
    before_err = np.concatenate((np.zeros_like(first)[:, None], errs[:, :-1]), axis=1)
    lam = np.zeros_like(first) if dh is None else np.asarray(dh, dtype=np.float64).copy()
    big, err = np.abs(lam), np.zeros_like(lam)
    lams, lam_errs = np.empty_like(x), np.empty_like(x)
    for t in range(x.shape[1] - 1, -1, -1):
        lam = dy[:, t] + lam
        big = np.abs(dy[:, t]) + big
        err = err + c[:, t] * big
        lams[:, t], lam_errs[:, t] = lam, err
        lam, big, err = a[:, t] * lam, a[:, t] * big, a[:, t] * (err + c[:, t] * big)
    slope = a if log else a * one_less
    inner = before - x if convex else before
    inner_err = before_err + (2.0 ** -24 * (np.abs(before) + np.abs(x)) if convex else 0.0)
    out = {"dx": w * lams, "dgate": lams * slope * inner, "d_initial_state": lam}
    bound = {"dx": w * (lam_errs + c * np.abs(lams)),
             "dgate": slope * (lam_errs * (np.abs(inner) + inner_err) + np.abs(lams) * inner_err
                               + 3 * c * np.abs(lams * inner)),
             "d_initial_state": err}
    return out, bound
