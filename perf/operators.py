"""Cases of the gated linear recurrence (whole sequences, their gradients, one
token) and of the layer norm (forward and gradients), for timing.

Each case names one operator, its sizes and its element type.  `run` makes one
pass: with `own` false through elementary torch operations in 32 bits, with
`own` true through this package's calls.

  recurrence  a = sigmoid(g) or exp(g);  h_t = a_t h_{t-1} + w_t x_t,
              w = 1 or (convex) 1 - a;  y_t = h_t
  layer norm  y = (x - mean) rstd weight + bias (rms: mean = 0), per row
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BLOCK = 256  # tokens between two saved states of a sequence
EPS = 1e-5


def listed():
    return [
        # the smallest scan workload of the library: launch latency
        dict(name="scan_tiny_f32", op="scan", dtype="f32", batch=1, len=256, channels=64, form="sigmoid",
             convex=False, resets=0, state=False),
        # prefill or training forward of a batch of ordinary sequences, continued from a state
        dict(name="scan_batch_bf16", op="scan", dtype="bf16", batch=8, len=2048, channels=2048, form="sigmoid",
             convex=True, resets=0, state=True),
        # one very long sequence: the time axis has to be split
        dict(name="scan_long_bf16", op="scan", dtype="bf16", batch=1, len=131072, channels=2048, form="sigmoid",
             convex=True, resets=0, state=False),
        # packed documents (the gate cuts the state at each start) of odd sizes
        dict(name="scan_ragged_f32", op="scan", dtype="f32", batch=3, len=1777, channels=1001, form="log",
             convex=False, resets=9, state=True),
        # training: gradients, with the states the forward call saved
        dict(name="backward_batch_bf16", op="backward", dtype="bf16", batch=8, len=2048, channels=2048,
             form="sigmoid", convex=True, resets=0, state=True, saved=True),
        # gradients of a few long sequences in full precision, nothing saved
        dict(name="backward_long_f32", op="backward", dtype="f32", batch=2, len=16384, channels=1000, form="log",
             convex=False, resets=4, state=False, saved=False),
        # generation for one sequence: launch latency
        dict(name="step_one_f32", op="step", dtype="f32", batch=1, channels=2048, form="log", convex=False),
        # generation for many sequences (the library's decode workload)
        dict(name="step_decode_bf16", op="step", dtype="bf16", batch=256, channels=5120, form="sigmoid",
             convex=True),
        # norm of one generated token per sequence
        dict(name="norm_tokens_bf16", op="norm", dtype="bf16", rows=256, channels=5120, rms=True, bias=False),
        # norm of a training batch's tokens
        dict(name="norm_batch_bf16", op="norm", dtype="bf16", rows=16384, channels=2048, rms=False, bias=True),
        # its gradients
        dict(name="norm_backward_batch_bf16", op="norm_backward", dtype="bf16", rows=16384, channels=2048,
             rms=False, bias=True),
        # gradients at odd sizes in full precision
        dict(name="norm_backward_ragged_f32", op="norm_backward", dtype="f32", rows=4099, channels=1001, rms=False,
             bias=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the listed kinds: 1 to 8 sequences of 1 to 131,072 tokens and
    1 to 5,120 channels (1 to 256 sequences in generation; up to 65,536 rows
    of 16 or more channels in a norm: with a few, a normed row is a constant
    and its gradient only rounding), never more elements than the largest
    listed scan or norm."""
    op = rng.choice(("scan", "scan", "backward", "backward", "step", "norm", "norm_backward"))
    case = dict(op=op, dtype=rng.choice(("f32", "bf16")))
    channels = _log_int(rng, 16 if op.startswith("norm") else 1, 5120)
    if rng.random() < 0.4:
        channels = max(8, channels // 8 * 8)
    case["channels"] = channels
    if op in ("norm", "norm_backward"):
        case["rows"] = _log_int(rng, 1, min(65536, (1 << 25) // channels))
        case["rms"] = rng.random() < 0.5
        case["bias"] = rng.random() < 0.5
        return case
    case["form"] = rng.choice(("sigmoid", "log"))
    case["convex"] = rng.random() < 0.5
    if op == "step":
        case["batch"] = _log_int(rng, 1, 256)
        return case
    case["batch"] = _log_int(rng, 1, 8)
    most = (1 << (25 if op == "backward" else 27)) // (channels * case["batch"])
    case["len"] = _log_int(rng, 1, min(131072, most))
    case["resets"] = rng.choice((0, 0, 5))
    case["state"] = rng.random() < 0.5
    if op == "backward":
        case["saved"] = rng.random() < 0.5
    return case


def _gates(case, shape, g, dtype):
    """Gate values of channels whose memory lasts between one and a thousand
    tokens, moved by the token; `resets` tokens per sequence (document starts)
    cut the state.  shape: (batch, len, channels)."""
    dev = dict(device="cuda", generator=g)
    memory = torch.exp(torch.rand(shape[2], **dev) * math.log(1000.0))
    gate = torch.randn(shape, **dev)
    if case["form"] == "sigmoid":
        gate = gate.add_(torch.log(memory))                # a / (1 - a) about memory
    else:
        gate = gate.mul_(0.5).exp_().div_(-memory)         # log a about -1 / memory
    gate = gate.to(dtype)
    if case.get("resets", 0):
        at = torch.randint(0, shape[1], (shape[0], case["resets"]), **dev)
        gate[torch.arange(shape[0], device="cuda")[:, None], at] = -math.inf
    return gate


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda", generator=g)
    dtype = DTYPES[case["dtype"]]
    ch = case["channels"]
    s = dict(case=case)
    if case["op"] in ("norm", "norm_backward"):
        rows = case["rows"]
        x = torch.randn((rows, ch), **dev)
        x = x.mul_(torch.rand((rows, 1), **dev) * 3 + 0.1).add_(torch.randn((rows, 1), **dev))
        s["x"] = x.to(dtype)
        s["weight"] = torch.randn(ch, **dev) * 0.2 + 1.0
        s["bias"] = torch.randn(ch, **dev) * 0.2 if case["bias"] else None
        if case["op"] == "norm_backward":
            s["dy"] = torch.randn((rows, ch), **dev).to(dtype)
            s["mean"], s["rstd"] = _row_statistics(s["x"].float(), case["rms"])  # what the forward call returned
        return s
    if case["op"] == "step":
        shape = (case["batch"], 1, ch)
        s["state"] = torch.randn((case["batch"], ch), **dev)
        s["x"] = torch.randn((case["batch"], ch), **dev).to(dtype)
        s["gate"] = _gates(case, shape, g, dtype)[:, 0].contiguous()
        return s
    shape = (case["batch"], case["len"], ch)
    s["x"] = torch.randn(shape, **dev).to(dtype)
    s["gate"] = _gates(case, shape, g, dtype)
    s["h0"] = torch.randn((case["batch"], ch), **dev) if case["state"] else None
    if case["op"] == "backward":
        s["dy"] = torch.randn(shape, **dev).to(dtype)
        s["dh"] = torch.randn((case["batch"], ch), **dev) if case["state"] else None
        s["checkpoints"] = None
        if case["saved"]:  # the state entering every block, as the forward call saved it
            a, w = _decay(s["gate"], case)
            h = _scan(a, _enter(a, w * s["x"].float(), s["h0"]))
            first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
            s["checkpoints"] = torch.cat((first, h[:, BLOCK - 1:-1:BLOCK]), 1).contiguous()
    return s


# --- plain forms -----------------------------------------------------------------

def _decay(gate, case):
    """a and w in 32 bits; 1 - a without cancellation."""
    g = gate.float()
    if case["form"] == "sigmoid":
        a = 1 / (1 + torch.exp(-g))
        w = 1 / (1 + torch.exp(g)) if case["convex"] else torch.ones_like(a)
    else:
        a = torch.exp(g)
        w = -torch.expm1(g) if case["convex"] else torch.ones_like(a)
    return a, w


def _enter(a, b, h0):
    """b with the entering state's part added to the first token."""
    if h0 is None:
        return b
    b[:, 0] += a[:, 0] * h0
    return b


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t along dimension 1, from zero: pairs of tokens
    are joined into one step, the half as long sequence is scanned, and the
    tokens in between follow from their neighbours."""
    n = a.shape[1]
    if n == 1:
        return b.clone()
    even, odd = slice(0, n - 1, 2), slice(1, n, 2)
    h = torch.empty_like(b)
    h[:, odd] = _scan(a[:, odd] * a[:, even], a[:, odd] * b[:, even] + b[:, odd])
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * h[:, 1:n - 1:2] + b[:, 2::2]
    return h


def _row_statistics(x, rms):
    mean = torch.zeros(x.shape[0], device=x.device) if rms else x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    return mean, 1 / torch.sqrt(var + EPS)


def _plain(s, case):
    op, x = case["op"], s["x"]
    if op == "norm":
        mean, rstd = _row_statistics(x.float(), case["rms"])
        y = (x.float() - mean[:, None]) * rstd[:, None] * s["weight"]
        y = y if s["bias"] is None else y + s["bias"]
        return dict(y=y.to(x.dtype), mean=mean, rstd=rstd)
    if op == "norm_backward":
        dy = s["dy"].float()
        xh = (x.float() - s["mean"][:, None]) * s["rstd"][:, None]
        dxh = dy * s["weight"]
        dx = dxh - xh * (dxh * xh).mean(1, keepdim=True)
        dx = dx if case["rms"] else dx - dxh.mean(1, keepdim=True)
        out = dict(dx=(dx * s["rstd"][:, None]).to(x.dtype), dweight=(dy * xh).sum(0))
        return out if s["bias"] is None else dict(out, dbias=dy.sum(0))
    a, w = _decay(s["gate"], case)
    if op == "step":
        s["state"].copy_(a * s["state"] + w * x.float())
        return dict(y=s["state"].to(x.dtype), state=s["state"])
    if op == "scan":
        h = _scan(a, _enter(a, w * x.float(), s["h0"]))
        return dict(y=h.to(x.dtype), final=h[:, -1].clone())
    # gradients: the adjoint is the same recurrence from the last token back,
    # with each token's gate taken from the token after it
    h = _scan(a, _enter(a, w * x.float(), s["h0"]))
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat((first, h[:, :-1]), 1)
    after = torch.cat((a[:, 1:], torch.ones_like(a[:, :1])), 1)
    dy = s["dy"].float()
    lam = _scan(after.flip(1), _enter(after.flip(1), dy.flip(1), s["dh"])).flip(1)
    da = lam * (before - x.float()) if case["convex"] else lam * before
    one_less = 1 / (1 + torch.exp(s["gate"].float())) if case["form"] == "sigmoid" else 1.0
    return dict(dx=(w * lam).to(x.dtype), dgate=(da * a * one_less).to(x.dtype),
                d_initial_state=a[:, 0] * lam[:, 0])


# --- the package's calls -----------------------------------------------------------

def _framework(s, case):
    from selective_state_space_29_b200 import mamba_ssm as m
    op = case["op"]
    if op == "norm":
        y, mean, rstd = m.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS, rms=case["rms"])
        return dict(y=y, mean=mean, rstd=rstd)
    if op == "norm_backward":
        g = m.layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], bias=s["bias"] is not None,
                                  rms=case["rms"])
        return {k: v for k, v in g.items() if v is not None}
    how = dict(gate_form=case["form"], convex=case["convex"])
    if op == "step":
        return dict(y=m.gated_step(s["state"], s["x"], s["gate"], **how), state=s["state"])
    if op == "scan":
        y, final = m.gated_scan(s["x"], s["gate"], initial_state=s["h0"], **how)
        return dict(y=y, final=final)
    return m.gated_scan_backward(s["x"], s["gate"], s["dy"], initial_state=s["h0"], d_final_state=s["dh"],
                                 checkpoints=s["checkpoints"], **how)


def run(state):
    return _framework(state, state["case"]) if own else _plain(state, state["case"])


def work(case):
    """Bytes: each input once, each output once.  Flops: the products, sums
    and elementary functions of the formulas."""
    es = 4 if case["dtype"] == "f32" else 2
    ch = case["channels"]
    if case["op"] in ("norm", "norm_backward"):
        n, rows = case["rows"] * ch, case["rows"]
        if case["op"] == "norm":
            return dict(bytes=2 * n * es + 8 * rows + 4 * ch * (2 if case["bias"] else 1), flops=8 * n)
        return dict(bytes=3 * n * es + 8 * rows + 4 * ch * (3 if case["bias"] else 2), flops=14 * n)
    rows = case["batch"] * ch
    extra = 3 if case["convex"] else 0
    if case["op"] == "step":
        return dict(bytes=rows * (8 + 3 * es), flops=rows * (6 + extra))
    n = rows * case["len"]
    if case["op"] == "scan":
        return dict(bytes=3 * n * es + 4 * rows * (2 if case["state"] else 1), flops=n * (6 + extra))
    blocks = -(-case["len"] // BLOCK)
    state = 4 * rows * ((2 if case["state"] else 0) + 1 + (blocks if case["saved"] else 0))
    return dict(bytes=5 * n * es + state, flops=n * (13 + extra))


# --- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = torch.float64
    x = s["x"].to(d)
    op = case["op"]
    if op in ("norm", "norm_backward"):
        n, wt = x.shape[1], s["weight"].to(d)
        if op == "norm":
            mean = x.sum(1) * (0.0 if case["rms"] else 1.0 / n)
            c = x - mean[:, None]
            rstd = ((c * c).sum(1) / n + EPS) ** -0.5
            y = c * rstd[:, None] * wt[None]
            return dict(y=y if s["bias"] is None else y + s["bias"].to(d), mean=mean, rstd=rstd)
        # y depends on x through c, and through rstd as d rstd = -rstd^3 sum(c dc) / n
        dy, r = s["dy"].to(d), s["rstd"].to(d)[:, None]
        c = x - s["mean"].to(d)[:, None]
        dc = dy * wt[None] * r - c * (r ** 3 / n) * (dy * wt[None] * c).sum(1, keepdim=True)
        dx = dc if case["rms"] else dc - dc.sum(1, keepdim=True) / n
        out = dict(dx=dx, dweight=(dy * c * r).sum(0))
        return out if s["bias"] is None else dict(out, dbias=dy.sum(0))
    g = s["gate"].to(d)
    a = torch.sigmoid(g) if case["form"] == "sigmoid" else torch.exp(g)
    b = x
    if case["convex"]:
        b = x * (torch.sigmoid(-g) if case["form"] == "sigmoid" else -torch.expm1(g))
    if op == "step":
        h = a * s["state"].to(d) + b
        return dict(y=h, state=h)
    length = case["len"]
    h = torch.zeros_like(b[:, 0]) if s["h0"] is None else s["h0"].to(d)
    h0, hs = h, torch.empty_like(b)
    for t in range(length):
        h = torch.addcmul(b[:, t], a[:, t], h, out=hs[:, t])
    if op == "scan":
        return dict(y=hs, final=hs[:, -1].clone())
    dy = s["dy"].to(d)
    lam = torch.zeros_like(h0) if s["dh"] is None else s["dh"].to(d)
    lams = torch.empty_like(b)
    for t in range(length - 1, -1, -1):
        after = lam if t == length - 1 else a[:, t + 1] * lam
        lam = torch.add(dy[:, t], after, out=lams[:, t])
    dx = lams if not case["convex"] else lams * (torch.sigmoid(-g) if case["form"] == "sigmoid" else -torch.expm1(g))
    prev = torch.cat((h0[:, None], hs[:, :-1]), 1)
    slope = a * torch.sigmoid(-g) if case["form"] == "sigmoid" else a
    dgate = lams * slope * (prev - x if case["convex"] else prev)
    return dict(dx=dx, dgate=dgate, d_initial_state=a[:, 0] * lams[:, 0])
