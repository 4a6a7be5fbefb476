"""Pins of the 64-bit oracles of the gated recurrence and the layer norm: closed
forms, and gradients against central differences."""
import numpy as np
import pytest

from oracle import gated, norm

RNG = np.random.default_rng(11)


def test_constant_gate_is_a_geometric_sum():
    a, n = 0.75, 40
    g = np.full((1, n, 1), np.log(a / (1 - a)))
    x = np.ones((1, n, 1))
    h, _ = gated.scan(x, g)
    np.testing.assert_allclose(h[0, :, 0], (1 - a ** np.arange(1, n + 1)) / (1 - a), rtol=1e-13)
    h, _ = gated.scan(x, np.full((1, n, 1), np.log(a)), log=True, convex=True)
    np.testing.assert_allclose(h[0, :, 0], 1 - a ** np.arange(1, n + 1), rtol=1e-13)


def test_unrolled_sum_and_reset():
    b, n, c = 2, 9, 3
    x, g, h0 = RNG.standard_normal((b, n, c)), RNG.standard_normal((b, n, c)), RNG.standard_normal((b, c))
    g[0, 4] = -np.inf
    for log in (False, True):
        gg = -np.abs(g) if log else g
        a, w, _ = gated.decay(gg, log, True)
        h, _ = gated.scan(x, gg, log, True, h0)
        for t in range(n):
            want = np.prod(a[:, :t + 1], axis=1) * h0
            for s in range(t + 1):
                want = want + np.prod(a[:, s + 1:t + 1], axis=1) * w[:, s] * x[:, s]
            np.testing.assert_allclose(h[:, t], want, rtol=1e-12, atol=1e-13)
        np.testing.assert_array_equal(h[0, 4], x[0, 4])


@pytest.mark.parametrize("log", [False, True])
@pytest.mark.parametrize("convex", [False, True])
def test_gated_gradients_against_differences(log, convex):
    b, n, c = 2, 7, 2
    x, dy = RNG.standard_normal((b, n, c)), RNG.standard_normal((b, n, c))
    g, h0, dh = RNG.standard_normal((b, n, c)), RNG.standard_normal((b, c)), RNG.standard_normal((b, c))
    if log:
        g = -np.exp(g)

    def loss(x, g, h0):
        h, _ = gated.scan(x, g, log, convex, h0)
        return (h * dy).sum() + (h[:, -1] * dh).sum()

    out, _ = gated.scan_backward(x, g, dy, log, convex, h0, dh)
    args = [x, g, h0]
    for i, name in enumerate(("dx", "dgate", "d_initial_state")):
        for at in np.ndindex(args[i].shape):
            up, down = [v.copy() for v in args], [v.copy() for v in args]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            # the difference's own error: rounding 2^-52 |loss| / 2e-6, and 1e-12 of its third derivative
            assert abs((loss(*up) - loss(*down)) / 2e-6 - out[name][at]) < 2e-8


@pytest.mark.parametrize("rms", [False, True])
def test_norm_gradients_against_differences(rms):
    rows, n, eps = 3, 5, 1e-3
    x, dy = RNG.standard_normal((rows, n)), RNG.standard_normal((rows, n))
    w, bias = RNG.standard_normal(n), RNG.standard_normal(n)

    def loss(x, w, bias):
        return (norm.layer_norm(x, w, bias, eps, rms)[0][0] * dy).sum()

    mean, rstd = norm.statistics(x, eps, rms)
    out, _ = norm.layer_norm_backward(dy, x, w, mean, rstd, rms)
    args = [x, w, bias]
    for i, name in enumerate(("dx", "dweight", "dbias")):
        for at in np.ndindex(args[i].shape):
            up, down = [v.copy() for v in args], [v.copy() for v in args]
            up[i][at] += 1e-6
            down[i][at] -= 1e-6
            assert abs((loss(*up) - loss(*down)) / 2e-6 - out[name][at]) < 2e-8


def test_norm_closed_form():
    (y, mean, rstd), _ = norm.layer_norm(np.array([[1.0, 3.0]]), None, None, 0.0)
    np.testing.assert_allclose(y, [[-1.0, 1.0]])
    assert mean[0] == 2.0 and rstd[0] == 1.0
    (y, _, rstd), _ = norm.layer_norm(np.array([[3.0, 4.0]]), np.array([2.0, 1.0]), None, 0.0, rms=True)
    np.testing.assert_allclose(y, [[6.0, 4.0]] / np.sqrt(12.5))


@pytest.mark.parametrize("log,convex", [(False, False), (False, True), (True, False), (True, True)])
def test_gated_bounds_hold_for_a_32_bit_evaluation(log, convex):
    """A plain float32 evaluation stays within the oracle's bounds, which are
    not so wide that they say nothing."""
    f = np.float32
    b, n, c = 2, 300, 8
    x = RNG.standard_normal((b, n, c)).astype(f)
    g = (RNG.standard_normal((b, n, c)) + 3).astype(f)
    if log:
        g = -np.exp(g - 6).astype(f)
    a = np.exp(g) if log else f(1) / (f(1) + np.exp(-g))
    w = (-np.expm1(g) if log else f(1) / (f(1) + np.exp(g))) if convex else np.ones_like(a)
    h = np.zeros((b, c), f)
    hs = np.empty_like(x)
    for t in range(n):
        h = a[:, t] * h + w[:, t] * x[:, t]
        hs[:, t] = h
    want, bound = gated.scan(x, g, log, convex)
    assert hs.dtype == f and (np.abs(hs - want) <= bound).all()
    assert bound.max() < 1e-2 * np.abs(want).max()
