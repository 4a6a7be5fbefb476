"""GPU tests of the layer norm and its gradients against the 64-bit oracle.
Tolerance per element: the oracle's bound of the 32-bit evaluation's error
(derived in oracle/norm.py) plus half a step of the element type, 2^-8 of the
value for bf16 and 2^-24 for float32.  Also: norms and recurrence together."""
import numpy as np
import pytest
import torch

from oracle import gated as gref
from oracle import norm as ref
from selective_state_space_29_b200 import mamba_ssm as m

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def check(name, got, want, bound):
    got_, tol = f64(got), bound + HALF_STEP[got.dtype] * (np.abs(want) + bound) + 1e-30
    assert np.isfinite(got_).all(), name
    worst = np.max(np.abs(got_ - want) - tol) if want.size else -1.0
    assert worst <= 0, f"{name}: {worst:.3e} over the tolerance"


def make(rows, channels, dtype, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=g)
    x = torch.randn((rows, channels), **kw) * (torch.rand((rows, 1), **kw) * 3 + 0.1) + torch.randn((rows, 1), **kw)
    return dict(x=x.to(dtype), dy=torch.randn((rows, channels), **kw).to(dtype),
                weight=1 + 0.3 * torch.randn(channels, **kw), bias=0.3 * torch.randn(channels, **kw))


def run_all(d, rms, weight=True, bias=True, eps=EPS):
    w, b = d["weight"] if weight else None, d["bias"] if bias else None
    y, mean, rstd = m.layer_norm(d["x"], w, b, eps=eps, rms=rms)
    (wy, wm, wr), (ey, em, er) = ref.layer_norm(f64(d["x"]), f64(w), f64(b), eps, rms)
    check("mean", mean, wm, em)
    check("rstd", rstd, wr, er)
    check("y", y, wy, ey)
    out = m.layer_norm_backward(d["dy"], d["x"], w, mean, rstd, bias=bias, rms=rms)
    want, bound = ref.layer_norm_backward(f64(d["dy"]), f64(d["x"]), f64(w), f64(mean), f64(rstd), rms)
    check("dx", out["dx"], want["dx"], bound["dx"])
    assert (out["dweight"] is None) == (not weight) and (out["dbias"] is None) == (not bias)
    for name in ("dweight", "dbias"):
        if out[name] is not None:
            check(name, out[name], want[name], bound[name])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("channels", [1, 2, 3, 5, 8, 16, 31, 32, 33, 63, 64, 65, 96, 127, 128, 130, 255, 256, 257, 511,
                                      512, 520, 1000, 1001, 1023, 1024, 1025, 2047, 2048, 2056, 4095, 4096, 5120,
                                      8191, 8192, 8200, 16383, 16384])
def test_channel_counts(channels, rms, dtype):
    run_all(make(7, channels, DT[dtype], seed=channels), rms)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,channels", [(1, 64), (2, 1001), (31, 48), (33, 200), (257, 72), (1000, 24), (601, 1024),
                                           (5000, 16), (20000, 8)])
def test_row_counts(rows, channels, dtype):
    run_all(make(rows, channels, DT[dtype], seed=rows), rows % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_without_weight_or_bias(weight, bias, dtype):
    run_all(make(40, 300, DT[dtype], seed=2), False, weight, bias)
    run_all(make(40, 296, DT[dtype], seed=2), True, weight, bias)


def test_rows_far_from_zero_and_constant_rows():
    """A mean a thousand times the spread; constant and zero rows (their
    variance is zero, so rstd = eps^-1/2)."""
    for channels in (64, 777, 2048):
        d = make(6, channels, torch.float32, seed=channels)
        d["x"] += 1000.0
        run_all(d, False)
        d["x"][1] = 3.0
        d["x"][2] = 0.0
        run_all(d, False)
        run_all(d, True)
        y, mean, rstd = m.layer_norm(d["x"], d["weight"], d["bias"])
        assert torch.equal(y[1], d["bias"]) and torch.equal(y[2], d["bias"])
        assert mean[1] == 3.0 and mean[2] == 0.0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("channels", [64, 1024, 5120])
def test_unaligned_pointers_and_untouched_neighbours(channels, offset, dtype):
    rows = 9
    d = make(rows, channels, DT[dtype], seed=offset)

    def inside(t, value=None):
        buf = torch.full((t.numel() + 64,), 7.0, device="cuda", dtype=t.dtype)
        view = buf[16 + offset:16 + offset + t.numel()].view(t.shape)
        if value is not None:
            view.copy_(value)
        return buf, view

    x, dy, w, b = (inside(d[k], d[k])[1] for k in ("x", "dy", "weight", "bias"))
    (yb, y), (xb, dx), (wb, dw), (bb, db) = inside(x), inside(x), inside(w), inside(w)
    code = m.dtype_code(x.dtype)
    mb, mean = inside(torch.empty(rows, device="cuda"))
    rb, rstd = inside(torch.empty(rows, device="cuda"))
    m.mamba_layer_norm(x, w, b, y, mean, rstd, rows, channels, EPS, 0, code)
    m.mamba_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, rows, channels, 0, code)
    (wy, wm, wr), (ey, em, er) = ref.layer_norm(f64(x), f64(w), f64(b), EPS)
    check("y", y, wy, ey)
    check("mean", mean, wm, em)
    check("rstd", rstd, wr, er)
    want, bound = ref.layer_norm_backward(f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
    for name, got in (("dx", dx), ("dweight", dw), ("dbias", db)):
        check(name, got, want[name], bound[name])
    for buf, view in ((yb, y), (xb, dx), (wb, dw), (bb, db), (mb, mean), (rb, rstd)):
        at = 16 + offset
        assert (buf[:at] == 7.0).all() and (buf[at + view.numel():] == 7.0).all()


def test_optional_outputs_and_empty_rows():
    d = make(12, 96, torch.bfloat16)
    x, dy, w = d["x"], d["dy"], d["weight"]
    y, mean, rstd = m.layer_norm(x, w)
    y2 = torch.empty_like(x)
    m.mamba_layer_norm(x, w, None, y2, None, None, 12, 96, EPS, 0, m.MAMBA_BF16)
    assert torch.equal(y, y2)
    out = m.layer_norm_backward(dy, x, w, mean, rstd)
    dx = torch.empty_like(x)
    m.mamba_layer_norm_backward(dy, x, w, mean, rstd, dx, None, None, 12, 96, 0, m.MAMBA_BF16)
    assert torch.equal(dx, out["dx"])
    db = torch.empty(96, device="cuda")
    m.mamba_layer_norm_backward(dy, x, w, mean, rstd, dx, None, db, 12, 96, 0, m.MAMBA_BF16)
    assert torch.equal(db, out["dbias"])
    # RMS: the mean is neither read nor needed
    y, mean, rstd = m.layer_norm(x, w, rms=True)
    assert (mean == 0).all()
    a = m.layer_norm_backward(dy, x, w, None, rstd, rms=True)
    b = m.layer_norm_backward(dy, x, w, torch.full_like(rstd, float("nan")), rstd, rms=True)
    assert all(torch.equal(a[k], b[k]) for k in a)
    e = torch.empty(0, 96, device="cuda")
    y, mean, rstd = m.layer_norm(e, w)
    assert y.shape == e.shape and mean.shape == (0,)
    out = m.layer_norm_backward(e, e, w, mean, rstd)
    assert (out["dweight"] == 0).all() and (out["dbias"] == 0).all() and out["dx"].shape == e.shape
    x3 = x.view(3, 4, 96)
    y, mean, rstd = m.layer_norm(x3, w)
    assert y.shape == x3.shape and mean.shape == (3, 4)
    assert torch.equal(y.view(12, 96), m.layer_norm(x, w)[0])


def test_helper_refusals():
    d = make(4, 32, torch.float32)
    x, w = d["x"], d["weight"]
    _, mean, rstd = m.layer_norm(x, w)
    for bad in (w[:31], w.bfloat16(), w.cpu(), torch.cat((w, w))[::2]):
        with pytest.raises(ValueError):
            m.layer_norm(x, bad)
        with pytest.raises(ValueError):
            m.layer_norm_backward(d["dy"], x, bad, mean, rstd)
    with pytest.raises(ValueError):
        m.layer_norm(x.t())
    with pytest.raises(ValueError):
        m.layer_norm(x.double())
    with pytest.raises(ValueError):
        m.layer_norm_backward(d["dy"][:3], x, w, mean, rstd)
    with pytest.raises(ValueError):
        m.layer_norm_backward(d["dy"], x, w, None, rstd)
    with pytest.raises(m.MambaError):
        m.layer_norm(x, w, y=x)
    with pytest.raises(m.MambaError):
        m.layer_norm(x, w, eps=-1.0)
    with pytest.raises(m.MambaError) as e:
        m.layer_norm(torch.zeros(2, m.MAMBA_NORM_MAX_CHANNELS + 1, device="cuda"))
    assert e.value.status == m.MAMBA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows,channels", [(40, 96), (40, 1001), (3000, 512), (40, 5120)])
def test_infinities_nan_and_squares_past_the_type(rows, channels, rms, dtype):
    """Rows that are not finite, or whose squares are not, give what the formula
    in 32 bits gives; the rows beside them are left alone."""
    d = make(rows, channels, DT[dtype], seed=31)
    y0, mean0, rstd0 = m.layer_norm(d["x"], d["weight"], d["bias"], eps=EPS, rms=rms)
    g0 = m.layer_norm_backward(d["dy"], d["x"], d["weight"], mean0, rstd0, rms=rms)
    x = d["x"].clone()
    x[3, 5], x[10, channels - 1], x[17, 0] = float("inf"), float("nan"), float("-inf")
    x[24] *= 1e25                                  # finite, its squares are not
    odd = torch.zeros(rows, dtype=torch.bool, device="cuda")
    odd[[3, 10, 17, 24]] = True
    y, mean, rstd = m.layer_norm(x, d["weight"], d["bias"], eps=EPS, rms=rms)
    assert torch.equal(y[~odd], y0[~odd]) and torch.equal(mean[~odd], mean0[~odd]) and torch.equal(rstd[~odd], rstd0[~odd])
    f = x[odd].float()
    want_mean = torch.zeros(4, device="cuda") if rms else f.mean(1)
    c = f - want_mean[:, None]
    want_rstd = (c.square().mean(1) + EPS).rsqrt()
    want = c * want_rstd[:, None] * d["weight"] + d["bias"]
    assert want_rstd[3] == 0 and want[1].isnan().all()
    assert torch.equal(mean[odd].isnan(), want_mean.isnan()) and torch.equal(mean[odd].isinf(), want_mean.isinf())
    assert torch.equal(rstd[odd].nan_to_num(-1.0), want_rstd.nan_to_num(-1.0))   # each 0 or NaN
    # where rstd is 0, y is the bias
    assert torch.equal(y[odd].nan_to_num(-1e9), want.to(x.dtype).nan_to_num(-1e9))
    g = m.layer_norm_backward(d["dy"], x, d["weight"], mean, rstd, rms=rms)
    assert torch.equal(g["dx"][~odd], g0["dx"][~odd])
    assert g["dx"][10].isnan().all() and (g["dx"][24] == 0).all()
    assert torch.equal(g["dbias"], g0["dbias"])


@pytest.mark.parametrize("rows,channels", [(3000, 256), (700, 2048), (40, 5120)])
def test_same_bits_every_call_streams_and_graphs(rows, channels):
    d = make(rows, channels, torch.bfloat16)
    y0, mean, rstd = m.layer_norm(d["x"], d["weight"], d["bias"])
    g0 = m.layer_norm_backward(d["dy"], d["x"], d["weight"], mean, rstd)
    other = make(rows + 5, channels, torch.bfloat16, seed=4)
    z, zm, zr = m.layer_norm(other["x"], other["weight"])
    o0 = m.layer_norm_backward(other["dy"], other["x"], other["weight"], zm, zr)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        o = m.layer_norm_backward(other["dy"], other["x"], other["weight"], zm, zr, stream=side)
        g = m.layer_norm_backward(d["dy"], d["x"], d["weight"], mean, rstd)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(g[k], g0[k]) for k in g) and all(torch.equal(o[k], o0[k]) for k in o)
    graphs, outs = [], []
    for src in (d, other):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y, mn, rs = m.layer_norm(src["x"], src["weight"], src["bias"])
            outs.append(m.layer_norm_backward(src["dy"], src["x"], src["weight"], mn, rs))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(outs[0][k], g0[k]) and torch.equal(outs[1][k], o0[k]) for k in g0)


def test_norm_recurrence_norm_forward_and_backward():
    """A block as a model trains it: norm, gate and value products, recurrence,
    norm; every gradient against the same chain of 64-bit oracles (in float32,
    whose products and roundings the tolerance counts), and the loss along one
    direction against its difference."""
    b, n, c = 2, 300, 48
    g = torch.Generator(device="cuda").manual_seed(21)
    kw = dict(device="cuda", generator=g)
    x = torch.randn((b, n, c), **kw)
    w1, b1 = 1 + 0.2 * torch.randn(c, **kw), 0.2 * torch.randn(c, **kw)
    w2 = 1 + 0.2 * torch.randn(c, **kw)
    wv, wg = torch.randn((c, c), **kw) / c ** 0.5, torch.randn((c, c), **kw) / c ** 0.5
    dz = torch.randn((b, n, c), **kw)
    y1, m1, r1 = m.layer_norm(x, w1, b1)
    v, gate = (y1.double() @ wv.double()).float(), (y1.double() @ wg.double() + 2).float()
    ckpt = m.gated_scan_checkpoints(v)
    h, _ = m.gated_scan(v, gate, convex=True, checkpoints=ckpt)
    z, m2, r2 = m.layer_norm(h, w2, rms=True)
    g2 = m.layer_norm_backward(dz, h, w2, m2, r2, bias=False, rms=True)
    gs = m.gated_scan_backward(v, gate, g2["dx"], checkpoints=ckpt, convex=True)
    dy1 = (gs["dx"].double() @ wv.double().t() + gs["dgate"].double() @ wg.double().t()).float()
    g1 = m.layer_norm_backward(dy1, x, w1, m1, r1)

    def chain(x, w1, b1, w2):
        (y1, _, _), _ = ref.layer_norm(x.reshape(-1, c), w1, b1, EPS)
        y1 = y1.reshape(b, n, c)
        h, _ = gref.scan(y1 @ f64(wv), y1 @ f64(wg) + 2, False, True)
        (z, mean, rstd), _ = ref.layer_norm(h.reshape(-1, c), w2, None, EPS, rms=True)
        return y1, h, z.reshape(b, n, c), rstd

    X, W1, B1, W2 = f64(x), f64(w1), f64(b1), f64(w2)
    ry1, rh, rz, rr2 = chain(X, W1, B1, W2)
    D = f64(dz)
    o2, _ = ref.layer_norm_backward(D.reshape(-1, c), rh.reshape(-1, c), W2, None, rr2, rms=True)
    os, _ = gref.scan_backward(ry1 @ f64(wv), ry1 @ f64(wg) + 2, o2["dx"].reshape(b, n, c), False, True)
    od = os["dx"] @ f64(wv).T + os["dgate"] @ f64(wg).T
    mu, rs = ref.statistics(X.reshape(-1, c), EPS)
    o1, _ = ref.layer_norm_backward(od.reshape(-1, c), X.reshape(-1, c), W1, mu, rs)
    # the chain's float32 roundings: about twenty of 2^-24 a value at each of four stages, each carried by factors
    # of order one and summed over memories of up to a hundred tokens: 4 * 20 * 100 * 2^-24 = 5e-4 of the root mean square
    for name, got, want in (("z", z, rz), ("dx", g1["dx"], o1["dx"].reshape(b, n, c)), ("dw1", g1["dweight"], o1["dweight"]),
                            ("db1", g1["dbias"], o1["dbias"]), ("dw2", g2["dweight"], o2["dweight"])):
        assert np.abs(f64(got) - want).max() <= 5e-4 * np.sqrt((want ** 2).mean()), name
    direction = [np.random.default_rng(i).standard_normal(a.shape) for i, a in enumerate((X, W1, B1, W2))]
    step = 1e-6
    up = (chain(*(a + step * d for a, d in zip((X, W1, B1, W2), direction)))[2] * D).sum()
    down = (chain(*(a - step * d for a, d in zip((X, W1, B1, W2), direction)))[2] * D).sum()
    along = sum((f64(got).reshape(d.shape) * d).sum()
                for got, d in zip((g1["dx"], g1["dweight"], g1["dbias"], g2["dweight"]), direction))
    size = sum(np.abs(f64(got).reshape(d.shape) * d).sum()
               for got, d in zip((g1["dx"], g1["dweight"], g1["dbias"], g2["dweight"]), direction))
    assert abs((up - down) / (2 * step) - along) <= 5e-4 * size


def test_norm_around_the_selective_scan():
    """The norm in front of the library's selective scan, with both backward passes."""
    from oracle import get
    b, n, c, s = 2, 130, 64, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    kw = dict(device="cuda", generator=g)
    x, w = torch.randn((b, n, c), **kw), 1 + 0.2 * torch.randn(c, **kw)
    delta = torch.rand((b, n, c), **kw) * 0.1 + 1e-3
    A = -(torch.arange(1, s + 1, device="cuda").float()).expand(c, s).contiguous()
    B, C = torch.randn((b, n, s), **kw), torch.randn((b, n, s), **kw)
    dy = torch.randn((b, n, c), **kw)
    u, mean, rstd = m.layer_norm(x, w, rms=True)
    m.selective_scan(u, delta, A, B, C)
    du = m.selective_scan_backward(u, delta, A, B, C, None, dy)["du"]
    out = m.layer_norm_backward(du, x, w, None, rstd, bias=False, rms=True)
    (ru, _, rr), _ = ref.layer_norm(f64(x).reshape(-1, c), f64(w), None, EPS, rms=True)
    grads = get().scan_backward(ru.reshape(b, n, c), f64(delta), f64(A), f64(B), f64(C), None, f64(dy))
    want, _ = ref.layer_norm_backward(grads["du"].reshape(-1, c), f64(x).reshape(-1, c), f64(w), None, rr, rms=True)
    # the selective scan's own float32 tolerance, 1e-4 of a row's largest value
    assert np.abs(f64(out["dx"]).reshape(-1, c) - want["dx"]).max() <= 1e-4 * np.abs(want["dx"]).max()
    assert np.abs(f64(out["dweight"]) - want["dweight"]).max() <= 1e-4 * np.abs(want["dweight"]).max()
