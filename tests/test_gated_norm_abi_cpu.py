"""Host-side checks of the gated recurrence's and the layer norm's entry points:
calls that are refused, or are no-ops, before any CUDA call; no GPU needed."""
import pytest

from selective_state_space_29_b200 import build as lib_build
from selective_state_space_29_b200 import mamba_ssm as m

KB = 1024


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return m.library()


def _call(fn, names, defaults):
    def call(**kw):
        a = dict(defaults)
        a.update(kw)
        return fn(*[a[n] for n in names], None)
    return call


@pytest.fixture(scope="module")
def scan(lib):
    names = ["x", "gate", "h0", "y", "fs", "ckpt", "batch", "len", "channels", "flags", "dtype"]
    return _call(lib.mamba_gated_scan, names,
                 dict(x=1 * KB, gate=2 * KB, h0=None, y=3 * KB, fs=None, ckpt=None, batch=1, len=4, channels=8,
                      flags=0, dtype=m.MAMBA_BF16))


@pytest.fixture(scope="module")
def backward(lib):
    names = ["x", "gate", "h0", "ckpt", "dy", "dh", "dx", "dgate", "dh0", "batch", "len", "channels", "flags", "dtype"]
    return _call(lib.mamba_gated_scan_backward, names,
                 dict(x=1 * KB, gate=2 * KB, h0=None, ckpt=None, dy=3 * KB, dh=None, dx=4 * KB, dgate=5 * KB,
                      dh0=None, batch=1, len=4, channels=8, flags=0, dtype=m.MAMBA_BF16))


@pytest.fixture(scope="module")
def step(lib):
    return _call(lib.mamba_gated_step, ["state", "x", "gate", "y", "batch", "channels", "flags", "dtype"],
                 dict(state=1 * KB, x=2 * KB, gate=3 * KB, y=4 * KB, batch=2, channels=8, flags=0,
                      dtype=m.MAMBA_BF16))


@pytest.fixture(scope="module")
def layer_norm(lib):
    names = ["x", "weight", "bias", "y", "mean", "rstd", "rows", "channels", "eps", "flags", "dtype"]
    return _call(lib.mamba_layer_norm, names,
                 dict(x=1 * KB, weight=2 * KB, bias=3 * KB, y=4 * KB, mean=5 * KB, rstd=6 * KB, rows=4, channels=8,
                      eps=1e-5, flags=0, dtype=m.MAMBA_BF16))


@pytest.fixture(scope="module")
def norm_backward(lib):
    names = ["dy", "x", "weight", "mean", "rstd", "dx", "dw", "db", "rows", "channels", "flags", "dtype"]
    return _call(lib.mamba_layer_norm_backward, names,
                 dict(dy=1 * KB, x=2 * KB, weight=3 * KB, mean=4 * KB, rstd=5 * KB, dx=6 * KB, dw=7 * KB, db=8 * KB,
                      rows=4, channels=8, flags=0, dtype=m.MAMBA_BF16))


INVALID, UNSUPPORTED, OK = m.MAMBA_ERR_INVALID_ARG, m.MAMBA_ERR_UNSUPPORTED, m.MAMBA_OK


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(batch=-1), dict(len=-1), dict(channels=-1), dict(flags=4),
                                dict(x=None), dict(gate=None), dict(y=None), dict(x=1025), dict(gate=2049),
                                dict(y=3073), dict(h0=1026), dict(fs=1026), dict(ckpt=1026),
                                dict(dtype=m.MAMBA_F32, x=1026),
                                dict(y=1 * KB), dict(y=1 * KB + 62), dict(y=2 * KB - 2),   # meets x, gate
                                dict(h0=8 * KB, fs=8 * KB), dict(fs=9 * KB, ckpt=9 * KB + 28)])
def test_scan_invalid(scan, kw):
    assert scan(**kw) == INVALID


def test_scan_sizes(scan):
    assert scan(batch=1 << 20, len=1 << 12) == UNSUPPORTED
    assert scan(batch=1 << 16, channels=1 << 16) == UNSUPPORTED
    assert scan(channels=1 << 31) == UNSUPPORTED
    assert scan(batch=1 << 62, len=4) == UNSUPPORTED        # no overflow on the way
    assert scan(batch=0) == OK and scan(channels=0) == OK
    assert scan(len=0) == OK and scan(len=0, x=None, gate=None, y=None) == OK


@pytest.mark.parametrize("kw", [dict(dtype=-1), dict(batch=-1), dict(len=-5), dict(channels=-1), dict(flags=8),
                                dict(x=None), dict(gate=None), dict(dy=None), dict(dx=None), dict(dgate=None),
                                dict(dx=4097), dict(dgate=5121), dict(dy=3073), dict(ckpt=1026), dict(dh=1026),
                                dict(dh0=1026), dict(dx=3 * KB), dict(dgate=4 * KB), dict(dx=1 * KB + 60),
                                dict(dh=9 * KB, dh0=9 * KB), dict(ckpt=9 * KB, dh0=9 * KB + 4)])
def test_backward_invalid(backward, kw):
    assert backward(**kw) == INVALID


def test_backward_sizes(backward):
    assert backward(batch=1 << 20, len=1 << 12) == UNSUPPORTED
    assert backward(batch=0) == OK and backward(channels=0) == OK
    assert backward(len=0) == OK


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(batch=-1), dict(channels=-1), dict(flags=4), dict(state=None),
                                dict(x=None), dict(gate=None), dict(y=None), dict(state=1026), dict(x=2049),
                                dict(y=2 * KB), dict(y=1 * KB), dict(y=3 * KB + 30), dict(state=2 * KB)])
def test_step_invalid(step, kw):
    assert step(**kw) == INVALID


def test_step_sizes(step):
    assert step(batch=0) == OK and step(channels=0) == OK
    assert step(batch=1 << 20, channels=1 << 12) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(rows=-1), dict(channels=-1), dict(flags=2), dict(eps=-1e-5),
                                dict(eps=float("nan")), dict(eps=float("inf")), dict(x=None), dict(y=None),
                                dict(x=1025), dict(weight=2050), dict(bias=3074), dict(mean=5122), dict(rstd=6146),
                                dict(y=1 * KB), dict(mean=2 * KB), dict(rstd=4 * KB), dict(rstd=5 * KB)])
def test_norm_invalid(layer_norm, kw):
    assert layer_norm(**kw) == INVALID


def test_norm_sizes(layer_norm):
    assert layer_norm(rows=0) == OK and layer_norm(channels=0) == OK
    assert layer_norm(channels=m.MAMBA_NORM_MAX_CHANNELS + 1) == UNSUPPORTED
    assert layer_norm(rows=1 << 31) == UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(rows=-1), dict(channels=-1), dict(flags=2), dict(dy=None),
                                dict(x=None), dict(dx=None), dict(rstd=None), dict(mean=None), dict(dy=1025),
                                dict(weight=3074), dict(dw=7170), dict(db=8194), dict(dx=1 * KB), dict(dx=2 * KB + 2),
                                dict(dw=3 * KB), dict(dw=8 * KB), dict(db=4 * KB)])
def test_norm_backward_invalid(norm_backward, kw):
    assert norm_backward(**kw) == INVALID


def test_norm_backward_sizes(norm_backward):
    assert norm_backward(channels=0) == OK
    assert norm_backward(rows=0, dw=None, db=None) == OK
    assert norm_backward(channels=m.MAMBA_NORM_MAX_CHANNELS + 1) == UNSUPPORTED
    assert norm_backward(rows=1 << 31) == UNSUPPORTED


def test_tensor_helpers_refuse_on_the_host():
    import torch
    x = torch.zeros(1, 2, 3)
    with pytest.raises(ValueError):
        m.gated_scan(x, x)                       # not CUDA tensors
    with pytest.raises(ValueError):
        m.gated_step(x[0], x[0], x[0])
    with pytest.raises(ValueError):
        m.layer_norm(x)
    with pytest.raises(ValueError):
        m._expect("t", torch.zeros(4, 6)[:, ::2], (4, 3), torch.float32, torch.device("cpu"))
    with pytest.raises(ValueError):
        m._expect("t", None, (4,), torch.float32, torch.device("cpu"))
    with pytest.raises(ValueError):
        m._expect("t", torch.zeros(4), (5,), torch.float32, torch.device("cpu"))
    with pytest.raises(ValueError):
        m._expect("t", torch.zeros(4), (4,), torch.bfloat16, torch.device("cpu"))
