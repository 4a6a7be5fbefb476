"""GPU tests of the gated recurrence (mamba_gated_scan, _backward, _step) against
the 64-bit oracle.  Tolerance per element: the oracle's bound of the 32-bit
evaluation's error (derived in oracle/gated.py) plus half a step of the
element type, 2^-8 of the value for bf16 and 2^-24 for float32, and 1e-30 for
products below the normal range."""
import numpy as np
import pytest
import torch

from oracle import gated as ref
from selective_state_space_29_b200 import mamba_ssm as m

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
FORMS = [("sigmoid", False), ("sigmoid", True), ("log", False), ("log", True)]


def f64(t):
    return t.detach().double().cpu().numpy()


def check(name, got, want, bound):
    got_, tol = f64(got), bound + HALF_STEP[got.dtype] * (np.abs(want) + bound) + 1e-30
    assert np.isfinite(got_).all(), name
    worst = np.max(np.abs(got_ - want) - tol) if want.size else -1.0
    assert worst <= 0, f"{name}: {worst:.3e} over the tolerance, at {np.unravel_index(np.argmax(np.abs(got_ - want) - tol), want.shape)}"


def make(batch, length, channels, dtype, form, seed=0, memory=300.0, resets=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    kw = dict(device="cuda", generator=g)
    shape = (batch, length, channels)
    tau = torch.exp(torch.rand(channels, **kw) * float(np.log(memory)))
    gate = torch.randn(shape, **kw)
    gate = gate + torch.log(tau) if form == "sigmoid" else -torch.exp(0.5 * gate) / tau
    gate = gate.to(dtype)
    for i in range(resets):
        at = int(torch.randint(0, length, (1,), **kw))
        gate[i % batch, at] = -float("inf") if i % 2 else torch.finfo(dtype).min
    d = dict(x=torch.randn(shape, **kw).to(dtype), gate=gate, dy=torch.randn(shape, **kw).to(dtype),
             h0=torch.randn((batch, channels), **kw), dh=torch.randn((batch, channels), **kw))
    return d


def run_all(d, form, convex, states=True, saved=True):
    """Forward and backward against the oracle."""
    h0, dh = (d["h0"], d["dh"]) if states else (None, None)
    n0 = None if h0 is None else f64(h0)
    nd = None if dh is None else f64(dh)
    log = form == "log"
    ckpt = m.gated_scan_checkpoints(d["x"]) if saved else None
    y, final = m.gated_scan(d["x"], d["gate"], initial_state=h0, gate_form=form, convex=convex, checkpoints=ckpt)
    h, e = ref.scan(f64(d["x"]), f64(d["gate"]), log, convex, n0)
    check("y", y, h, e)
    check("final", final, h[:, -1], e[:, -1])
    if saved:
        first = np.zeros_like(h[:, :1]) if n0 is None else n0[:, None]
        check("checkpoints", ckpt, np.concatenate((first, h[:, 255:-1:256]), 1),
              np.concatenate((np.zeros_like(first), e[:, 255:-1:256]), 1))
    out = m.gated_scan_backward(d["x"], d["gate"], d["dy"], initial_state=h0, d_final_state=dh, checkpoints=ckpt,
                                gate_form=form, convex=convex)
    want, bound = ref.scan_backward(f64(d["x"]), f64(d["gate"]), f64(d["dy"]), log, convex, n0, nd)
    for name in want:
        check(name, out[name], want[name], bound[name])
    assert m.mamba_get_device_error() == m.MAMBA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form,convex", FORMS)
@pytest.mark.parametrize("shape", [(1, 1, 1), (2, 2, 3), (1, 255, 33), (2, 256, 64), (2, 257, 31), (3, 600, 66),
                                   (1, 1500, 130), (2, 31, 200), (1, 4100, 8)])
def test_against_oracle(shape, form, convex, dtype):
    d = make(*shape, DT[dtype], form, seed=sum(shape))
    run_all(d, form, convex, states=shape[0] != 2, saved=shape[1] % 2 == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("channels", [1, 2, 4, 6, 7, 8, 16, 24, 63, 64, 65, 72, 127, 128, 129, 256, 257, 1001])
def test_channel_counts(channels, dtype):
    d = make(2, 300, channels, DT[dtype], "sigmoid", seed=channels, resets=3)
    run_all(d, "sigmoid", True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("length", [1, 2, 3, 7, 8, 9, 15, 16, 17, 32, 33, 63, 64, 65, 127, 128, 129, 511, 512, 513, 769])
def test_lengths(length, dtype):
    d = make(2, length, 40, DT[dtype], "log", seed=length, resets=2)
    run_all(d, "log", False, saved=length % 2 == 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form,convex", FORMS)
def test_resets_and_extreme_gates(form, convex, dtype):
    d = make(3, 700, 48, DT[dtype], form, seed=5, resets=12)
    gate = d["gate"]
    gate[0, 256:512] = -float("inf")              # a block with nothing kept
    gate[1, 0] = -float("inf")                    # nothing of the initial state
    gate[1, 699] = torch.finfo(gate.dtype).min
    gate[2, 100:300, ::3] = 0.0                   # log form: nothing decays
    gate[2, 300:310] = -200.0                     # below the smallest float
    gate[2, 310:320] = -85.0
    if form == "sigmoid":
        gate[2, 320:330] = 200.0
        gate[2, 330:340, 1] = float("inf")
        gate[2, 340:350] = 85.0
    run_all(d, form, convex)
    run_all(d, form, convex, saved=False)
    y, _ = m.gated_scan(d["x"], gate, initial_state=d["h0"], gate_form=form, convex=convex)
    assert torch.equal(y[0, 256:512], d["x"][0, 256:512]) and torch.equal(y[1, 0], d["x"][1, 0])
    out = m.gated_scan_backward(d["x"], gate, d["dy"], initial_state=d["h0"], d_final_state=d["dh"], gate_form=form,
                                convex=convex)
    assert (out["dgate"][0, 256:512] == 0).all() and (out["d_initial_state"][1] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_long_sequence_long_memory(dtype):
    """Memories of up to 20,000 tokens over 30,001 tokens: what enters the
    first blocks reaches the last ones."""
    d = make(1, 30001, 5, DT[dtype], "log", seed=3, memory=20000.0)
    run_all(d, "log", False)
    run_all(d, "log", True, saved=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_unaligned_pointers_and_untouched_neighbours(offset, dtype):
    """Tensors that start `offset` elements after an aligned address, inside
    larger buffers whose other elements stay as they were."""
    b, n, c = 2, 300, 64
    d = make(b, n, c, DT[dtype], "sigmoid", seed=offset)
    numel = b * n * c

    def inside(t, value=None):
        buf = torch.full((t.numel() + 2 * 64,), 77.0, device="cuda", dtype=t.dtype)
        view = buf[64 + offset - 8:64 + offset - 8 + t.numel()].view(t.shape)
        if value is not None:
            view.copy_(value)
        return buf, view

    x, gate, dy = (inside(d[k], d[k])[1] for k in ("x", "gate", "dy"))
    (yb, y), (db, dx), (gb, dg) = inside(x), inside(x), inside(x)
    fb, final = inside(d["h0"])
    cb, ckpt = inside(m.gated_scan_checkpoints(d["x"]))
    hb, dh0 = inside(d["h0"])
    m.gated_scan(x, gate, initial_state=d["h0"], convex=True, checkpoints=ckpt, y=y, final_state=final)
    m.mamba_gated_scan_backward(x, gate, d["h0"], ckpt, dy, d["dh"], dx, dg, dh0, b, n, c, m.MAMBA_GATE_CONVEX,
                                m.dtype_code(x.dtype))
    y2, final2 = m.gated_scan(d["x"], d["gate"], initial_state=d["h0"], convex=True)
    h, e = ref.scan(f64(x), f64(gate), False, True, f64(d["h0"]))
    check("y", y, h, e)
    check("y2", y2, h, e)
    check("final", final, h[:, -1], e[:, -1])
    want, bound = ref.scan_backward(f64(x), f64(gate), f64(dy), False, True, f64(d["h0"]), f64(d["dh"]))
    for name, got in (("dx", dx), ("dgate", dg), ("d_initial_state", dh0)):
        check(name, got, want[name], bound[name])
    for buf, view in ((yb, y), (db, dx), (gb, dg), (fb, final), (cb, ckpt), (hb, dh0)):
        buf = buf.clone()
        at = 64 + offset - 8
        buf[at:at + view.numel()] = 77.0
        assert (buf == 77.0).all()


@pytest.mark.parametrize("shape", [(1, 20000, 64), (2, 3000, 300), (8, 700, 1024)])
def test_same_bits_every_call_and_with_other_work_beside(shape):
    d = make(*shape, torch.bfloat16, "sigmoid", seed=9)
    other = make(2, 5000, 96, torch.float32, "log", seed=10)
    ckpt = m.gated_scan_checkpoints(d["x"])
    y0, f0 = m.gated_scan(d["x"], d["gate"], checkpoints=ckpt)
    g0 = m.gated_scan_backward(d["x"], d["gate"], d["dy"], checkpoints=ckpt)
    z0, _ = m.gated_scan(other["x"], other["gate"], gate_form="log")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        z, _ = m.gated_scan(other["x"], other["gate"], gate_form="log", stream=side)
        y, f = m.gated_scan(d["x"], d["gate"])
        g = m.gated_scan_backward(d["x"], d["gate"], d["dy"])
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(y, y0) and torch.equal(f, f0) and torch.equal(z, z0)
        for k in g:
            assert torch.equal(g[k], g0[k]), k


def test_empty_and_partial_outputs():
    h0 = torch.randn(2, 8, device="cuda")
    x = torch.empty(2, 0, 8, device="cuda")
    y, f = m.gated_scan(x, x, initial_state=h0)
    assert y.shape == x.shape and torch.equal(f, h0)
    _, f = m.gated_scan(x, x)
    assert (f == 0).all()
    out = m.gated_scan_backward(x, x, x, d_final_state=h0)
    assert torch.equal(out["d_initial_state"], h0)
    for shape in ((0, 5, 8), (2, 5, 0)):
        x = torch.empty(shape, device="cuda")
        y, f = m.gated_scan(x, x)
        assert y.shape == x.shape and f.shape == (shape[0], shape[2])
        m.gated_scan_backward(x, x, x)
    d = make(1, 300, 8, torch.float32, "log", seed=1)
    y, f = m.gated_scan(d["x"], d["gate"], gate_form="log", return_final_state=False)
    assert f is None
    assert torch.equal(y, m.gated_scan(d["x"], d["gate"], gate_form="log")[0])
    # the initial state's gradient is not wanted
    dx, dg = torch.empty_like(y), torch.empty_like(y)
    m.mamba_gated_scan_backward(d["x"], d["gate"], None, None, d["dy"], None, dx, dg, None, 1, 300, 8,
                                m.MAMBA_GATE_LOG, m.MAMBA_F32)
    out = m.gated_scan_backward(d["x"], d["gate"], d["dy"], gate_form="log")
    assert torch.equal(dx, out["dx"]) and torch.equal(dg, out["dgate"])


def test_helper_refusals():
    d = make(2, 6, 8, torch.float32, "sigmoid")
    x, g = d["x"], d["gate"]
    for bad in (g.bfloat16(), g[:, :5], g[:, :, :7], g.cpu(), g.transpose(1, 2)):
        with pytest.raises(ValueError):
            m.gated_scan(x, bad)
        with pytest.raises(ValueError):
            m.gated_scan_backward(x, g, bad)
    with pytest.raises(ValueError):
        m.gated_scan(x.half(), g.half())
    with pytest.raises(ValueError):
        m.gated_scan(x, g, initial_state=d["h0"].bfloat16())
    with pytest.raises(ValueError):
        m.gated_scan(x, g, checkpoints=torch.empty(2, 2, 8, device="cuda"))
    with pytest.raises(KeyError):
        m.gated_scan(x, g, gate_form="tanh")
    with pytest.raises(m.MambaError):
        m.gated_scan(x, g, y=x)
    with pytest.raises(m.MambaError):
        m.gated_scan(x, g, initial_state=d["h0"], final_state=d["h0"])
    with pytest.raises(ValueError):
        m.gated_step(d["h0"], x[:, 0], g[:, 0])     # rows of another tensor: not contiguous


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("form,convex", FORMS)
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (2, 64), (5, 1001), (256, 520)])
def test_steps_follow_the_scan(shape, form, convex, dtype):
    """Prefill, then tokens one by one from its final state: each step against
    the oracle's scan of the whole sequence."""
    b, c = shape
    d = make(b, 12, c, DT[dtype], form, seed=b + c, resets=2)
    d["gate"][:, 9] = -float("inf")
    _, state = m.gated_scan(d["x"][:, :4].contiguous(), d["gate"][:, :4].contiguous(), initial_state=d["h0"],
                            gate_form=form, convex=convex)
    h, e = ref.scan(f64(d["x"]), f64(d["gate"]), form == "log", convex, f64(d["h0"]))
    for t in range(4, 12):
        y = m.gated_step(state, d["x"][:, t].contiguous(), d["gate"][:, t].contiguous(), gate_form=form, convex=convex)
        check("y", y, h[:, t], e[:, t])
        check("state", state, h[:, t], e[:, t])


@pytest.mark.parametrize("offset", [1, 2, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_step_unaligned_and_untouched_neighbours(offset, dtype):
    b, c = 3, 40
    d = make(b, 1, c, DT[dtype], "sigmoid", seed=offset)
    sb = torch.full((b * c + 64,), 5.0, device="cuda")
    state = sb[16 + offset:16 + offset + b * c].view(b, c)
    state.copy_(d["h0"])
    yb = torch.full((b * c + 64,), 5.0, device="cuda", dtype=DT[dtype])
    y = yb[16 + offset:16 + offset + b * c].view(b, c)
    xb = torch.empty(b * c + 64, device="cuda", dtype=DT[dtype])
    x = xb[offset:offset + b * c].view(b, c)
    x.copy_(d["x"][:, 0])
    m.gated_step(state, x, d["gate"][:, 0].contiguous(), y=y)
    h, e = ref.scan(f64(d["x"]), f64(d["gate"]), False, False, f64(d["h0"]))
    check("y", y, h[:, 0], e[:, 0])
    check("state", state, h[:, 0], e[:, 0])
    for buf in (sb, yb):
        assert (buf[:16 + offset] == 5.0).all() and (buf[16 + offset + b * c:] == 5.0).all()


def test_captured_graphs_replayed_with_new_inputs():
    """Forward and backward in one graph, a step in another, replayed on new
    inputs, in turn, and beside eager calls of the same buffers."""
    d = make(2, 1500, 96, torch.bfloat16, "sigmoid", seed=1)
    bufs = {k: v.clone() for k, v in d.items()}
    state = torch.zeros_like(d["h0"])

    def once():
        ckpt = m.gated_scan_checkpoints(bufs["x"])
        y, f = m.gated_scan(bufs["x"], bufs["gate"], initial_state=bufs["h0"], checkpoints=ckpt)
        g = m.gated_scan_backward(bufs["x"], bufs["gate"], bufs["dy"], checkpoints=ckpt)
        g2 = m.gated_scan_backward(bufs["x"], bufs["gate"], bufs["dy"], initial_state=bufs["h0"])
        return [y, f, *g.values(), *g2.values()]

    def token():
        return m.gated_step(state, bufs["x"][:, 0].contiguous(), bufs["gate"][:, 0].contiguous())

    once(), token()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for fn in (once, once, token):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(fn())
        graphs.append(graph)
    for seed in (2, 3):
        new = make(2, 1500, 96, torch.bfloat16, "sigmoid", seed=seed)
        for k in bufs:
            bufs[k].copy_(new[k])
        graphs[0].replay()
        graphs[1].replay()
        want = once()
        graphs[0].replay()
        torch.cuda.synchronize()
        for got in outs[:2]:
            for a, b in zip(got, want):
                assert torch.equal(a, b)
        h, e = ref.scan(f64(new["x"]), f64(new["gate"]), False, False, f64(new["h0"]))
        check("y", outs[0][0], h, e)
        before = state.clone()
        graphs[2].replay()
        again = before
        y = m.gated_step(again, new["x"][:, 0].contiguous(), new["gate"][:, 0].contiguous())
        assert torch.equal(state, again) and torch.equal(outs[2], y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 16384, 1000), (1, 9000, 2048), (8, 2048, 512), (3, 2500, 333), (40, 300, 72)])
def test_no_wait_runs_out_over_many_calls(shape, dtype):
    """Many calls of many tiles a CTA, the last ones among them: the warps of a
    CTA hand barriers on without losing a phase, and every call gives the same bits."""
    d = make(*shape, DT[dtype], "log", seed=4)
    first = None
    for _ in range(25):
        y, f = m.gated_scan(d["x"], d["gate"], gate_form="log", convex=True)
        g = m.gated_scan_backward(d["x"], d["gate"], d["dy"], gate_form="log", convex=True)
        got = [y, f, *g.values()]
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))
    assert m.mamba_get_device_error() == m.MAMBA_OK


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_and_nan_stay_in_their_channel(dtype):
    """Values outside the contract: other channels and earlier tokens are as
    they would be without them, every call gives the same, and no wait runs out."""
    d = make(2, 1100, 72, DT[dtype], "sigmoid", seed=6)
    y0, _ = m.gated_scan(d["x"], d["gate"])
    g0 = m.gated_scan_backward(d["x"], d["gate"], d["dy"])
    bad = {k: v.clone() for k, v in d.items()}
    bad["x"][0, 300, 3], bad["x"][1, 700, 40] = float("nan"), float("inf")
    bad["gate"][0, 10, 5], bad["gate"][1, 1099, 71] = float("nan"), float("nan")
    bad["dy"][0, 500, 7] = float("-inf")
    y, _ = m.gated_scan(bad["x"], bad["gate"])
    g = m.gated_scan_backward(bad["x"], bad["gate"], bad["dy"])
    keep = torch.ones(2, 72, dtype=torch.bool, device="cuda")
    keep[0, [3, 5, 7]] = False
    keep[1, [40, 71]] = False
    for a, b in ((y, y0), (g["dx"], g0["dx"]), (g["dgate"], g0["dgate"])):
        assert torch.equal(a.transpose(1, 2)[keep], b.transpose(1, 2)[keep])
    assert torch.equal(y[0, :300, 3], y0[0, :300, 3]) and y[0, 300:512, 3].isnan().all()
    assert torch.equal(g["dx"][0, 501:, 7], g0["dx"][0, 501:, 7])
    assert torch.equal(g["d_initial_state"][keep], g0["d_initial_state"][keep])
    for _ in range(5):
        again = m.gated_scan_backward(bad["x"], bad["gate"], bad["dy"])
        for k in g:
            assert torch.equal(again[k].isnan(), g[k].isnan())
            assert torch.equal(again[k].nan_to_num(0.0, 1.0, -1.0), g[k].nan_to_num(0.0, 1.0, -1.0))
    assert m.mamba_get_device_error() == m.MAMBA_OK


def test_waits_are_full_length_after_an_old_error():
    """A timeout left on record by an earlier call changes nothing."""
    d = make(1, 5000, 64, torch.bfloat16, "log", seed=2)
    y0, f0 = m.gated_scan(d["x"], d["gate"], gate_form="log")
    m.mamba_debug_expire_wait(2_000_000)
    y, f = m.gated_scan(d["x"], d["gate"], gate_form="log")
    assert torch.equal(y, y0) and torch.equal(f, f0)
    assert m.mamba_get_device_error(clear=True) == m.MAMBA_ERR_TIMEOUT
    assert m.mamba_get_device_error() == m.MAMBA_OK
