"""The layer operators around a scan: the short causal convolution, the selective scan with one decay per channel
and state entry, and the layer norm (binding of the ssd_conv_*, ssd_selective_* and ssd_layer_norm_* entries of
include/ssd.h; argument marshalling only).

x, dt, z, B, C and the convolution's states are bfloat16, float16 or float32, one type per call; weights, A, D, the
scan's states and every summed gradient are float32.  Inputs may be column slices of a wider tensor: only the last
dimension has to be dense.  ``lengths`` (batch,) int32 says how many tokens of each row count, ``slots`` (batch,)
int32 which state of a pool each row works on (negative: an idle row).  ``stream`` is a torch.cuda.Stream (default:
the current one); outputs are allocated on it.
"""
from __future__ import annotations

import ctypes

import torch

from . import _ffi

_TYPES = {torch.bfloat16: _ffi.SSD_BF16, torch.float16: _ffi.SSD_F16, torch.float32: _ffi.SSD_F32}
_f32, _i32 = torch.float32, torch.int32


class _Launch:
    """The call's stream: made the current one while outputs are allocated and the library launches."""

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        if self.stream is None:
            return torch.cuda.current_stream().cuda_stream
        self.context = torch.cuda.stream(self.stream)
        self.context.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.stream is not None:
            self.context.__exit__(*exc)
        return False


def _dtype(t, name):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    code = _TYPES.get(t.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {t.dtype}")
    return code


def _check(t, name, dtype, shape, like):
    """A CUDA tensor of this type and shape, on `like`'s device and on the current one."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != like.get_device():
        raise ValueError(f"{name} must be on {like.device}, got {t.device}")


def _dense(t, name, dtype, shape, like):
    """The address of a dense tensor; None for None."""
    if t is None:
        return None
    _check(t, name, dtype, shape, like)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _strides(t, name, inner):
    """The strides of the dimensions before the last `inner`, which have to be dense; 0 for a dimension of one."""
    size, stride = t.shape, t.stride()
    need = 1
    for d in range(len(size) - 1, len(size) - 1 - inner, -1):
        if size[d] != 1 and stride[d] != need:
            raise ValueError(f"the last {inner} dimension(s) of {name} must be dense, got strides {stride}")
        need *= size[d]
    return [0 if size[d] == 1 else stride[d] for d in range(len(size) - inner)]


def _rows(t, name, dtype, shape, like, inner=1):
    """The address and strides of a tensor of rows; zeros for None."""
    if t is None:
        return None, [0] * (len(shape) - inner)
    _check(t, name, dtype, shape, like)
    return t.data_ptr(), _strides(t, name, inner)


def _input(t, name, ndim):
    code = _dtype(t, name)
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return code


def _keep(stream, *tensors):
    """Tells the allocator that `stream` uses these tensors, which may belong to another one."""
    if stream is not None:
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


def _conv_sizes(weight, channels, x):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a (channels, width) tensor")
    return weight.shape[1], _dense(weight, "weight", _f32, (channels, weight.shape[1]), x)


def _split(splits, channels):
    parts = [channels] if splits is None else [int(n) for n in splits]
    if not 1 <= len(parts) <= 3 or min(parts) < 1 or sum(parts) != channels:
        raise ValueError(f"splits must be one to three positive sizes that add up to {channels}, got {splits}")
    return parts


def _flat(ptrs, parts):
    out = []
    for i in range(3):
        out += [ptrs[i], parts[i]] if i < len(parts) else [None, 0]
    return out


def ssd_conv_forward(x, weight, bias=None, init_state=None, lengths=None, silu=True, splits=None, want_final=True,
                     stream=None):
    """Short causal depthwise convolution -> (y, final_state or None).

    x (batch, L, channels), weight (channels, width) f32 with width 2 to 4, bias (channels,) f32 or None, init_state
    (batch, width - 1, channels) or None.  y is (batch, L, channels), or with ``splits`` a tuple of dense tensors of
    those numbers of channels (a scan's x, B and C); final_state is the row's last width - 1 inputs."""
    code = _input(x, "x", 3)
    b, L, ch = x.shape
    W, wp = _conv_sizes(weight, ch, x)
    bp = _dense(bias, "bias", _f32, (ch,), x)
    ip = _dense(init_state, "init_state", x.dtype, (b, W - 1, ch), x)
    lp = _dense(lengths, "lengths", _i32, (b,), x)
    xb, xt = _strides(x, "x", 1)
    parts = _split(splits, ch)
    with _Launch(stream) as s:
        y = [x.new_empty((b, L, n)) for n in parts]
        final = x.new_empty((b, W - 1, ch)) if want_final else None
        _ffi.check("ssd_conv_forward", _ffi.lib().ssd_conv_forward(
            code, x.data_ptr(), xb, xt, wp, bp, ip, lp, b, L, ch, W, bool(silu),
            *_flat([v.data_ptr() for v in y], parts), None if final is None else final.data_ptr(), s))
    _keep(stream, x, weight, bias, init_state, lengths)
    return (y[0] if splits is None else tuple(y)), final


def ssd_conv_backward(x, weight, bias, dy, init_state=None, lengths=None, silu=True, dfinal=None, dx=None,
                      want_dinit=False, stream=None):
    """Gradients through ssd_conv_forward -> dict of dx, dweight (channels, width) f32, dbias (channels,) f32 (None
    without a bias), dinit (None unless wanted).

    dy is one tensor or the tuple of pieces, each dense and of x's type or float32; dfinal is the gradient of the
    final state.  ``dx`` may be given: a tensor like x whose last dimension is dense (a slice of a projection's
    gradient)."""
    code = _input(x, "x", 3)
    b, L, ch = x.shape
    W, wp = _conv_sizes(weight, ch, x)
    bp = _dense(bias, "bias", _f32, (ch,), x)
    ip = _dense(init_state, "init_state", x.dtype, (b, W - 1, ch), x)
    lp = _dense(lengths, "lengths", _i32, (b,), x)
    fp = _dense(dfinal, "dfinal", x.dtype, (b, W - 1, ch), x)
    xb, xt = _strides(x, "x", 1)
    pieces = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    parts = _split([p.shape[-1] for p in pieces], ch)
    flat = []
    for i in range(3):
        if i < len(parts):
            p = pieces[i]
            kind = _f32 if p.dtype == _f32 else x.dtype
            flat += [_dense(p, f"dy[{i}]", kind, (b, L, parts[i]), x), parts[i], p.dtype == _f32]
        else:
            flat += [None, 0, 0]
    with _Launch(stream) as s:
        if dx is None:
            dx = x.new_empty((b, L, ch))
        op, (ob, ot) = _rows(dx, "dx", x.dtype, (b, L, ch), x)
        dweight = x.new_empty((ch, W), dtype=_f32)
        dbias = x.new_empty((ch,), dtype=_f32) if bias is not None else None
        dinit = x.new_empty((b, W - 1, ch)) if want_dinit else None
        _ffi.check("ssd_conv_backward", _ffi.lib().ssd_conv_backward(
            code, x.data_ptr(), xb, xt, wp, bp, ip, lp, b, L, ch, W, bool(silu), *flat, fp, op, ob, ot,
            dweight.data_ptr(), None if dbias is None else dbias.data_ptr(),
            None if dinit is None else dinit.data_ptr(), s))
    _keep(stream, x, weight, bias, init_state, lengths, dfinal, dx, *pieces)
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dinit": dinit}


def _pool(state, slots, batch, shape, dtype, like):
    """The addresses of the states and the slots, and the number of states."""
    if not isinstance(state, torch.Tensor) or state.dim() != len(shape) + 1:
        raise ValueError(f"state must be (slots, {', '.join(map(str, shape))})")
    n = state.shape[0]
    if slots is None and n < batch:
        raise ValueError(f"state holds {n} rows for a batch of {batch}")
    return _dense(state, "state", dtype, (n, *shape), like), _dense(slots, "slots", _i32, (batch,), like), n


def ssd_conv_step(x, weight, bias, state, slots=None, silu=True, splits=None, stream=None):
    """ssd_conv_forward for one token of every row -> y (batch, channels), or the tuple of pieces.

    x (batch, channels); state (nslots, width - 1, channels) of x's type, updated in place."""
    code = _input(x, "x", 2)
    b, ch = x.shape
    W, wp = _conv_sizes(weight, ch, x)
    bp = _dense(bias, "bias", _f32, (ch,), x)
    sp, lp, n = _pool(state, slots, b, (W - 1, ch), x.dtype, x)
    (xb,) = _strides(x, "x", 1)
    parts = _split(splits, ch)
    with _Launch(stream) as s:
        y = [x.new_empty((b, m)) for m in parts]
        _ffi.check("ssd_conv_step", _ffi.lib().ssd_conv_step(
            code, x.data_ptr(), xb, wp, bp, sp, lp, n, b, ch, W, bool(silu), *_flat([v.data_ptr() for v in y], parts), s))
    _keep(stream, x, weight, bias, state, slots)
    return y[0] if splits is None else tuple(y)


def _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, rows):
    """What the three entries share: the element type, the leading arguments, strides, options and sizes."""
    code = _input(x, "x", len(rows) + 1)
    ch, T = x.shape[-1], x.dtype
    if not isinstance(B, torch.Tensor) or B.dim() != len(rows) + 2:
        raise ValueError(f"B must have {len(rows) + 2} dims (..., ngroups, dstate)")
    G, N = B.shape[-2:]
    if G < 1 or ch % G:
        raise ValueError(f"ngroups ({G}) must divide channels ({ch})")
    bc = (*rows, G, N)
    ptr, st = {}, []
    for name, t, shape, inner in (("x", x, x.shape, 1), ("dt", dt, x.shape, 1), ("z", z, x.shape, 1), ("B", B, bc, 2),
                                  ("C", C, bc, 2)):
        if t is None and name != "z":
            raise ValueError(f"{name} is required")
        ptr[name], s = _rows(t, name, T, shape, x, inner)
        st += s if len(rows) == 2 else [s[0], 0]
    o = _ffi.InputOptions(_dense(dt_bias, "dt_bias", _f32, (ch,), x), bool(dt_softplus), 0, 0.0, 0.0, 0, ptr["z"])
    if dt_limit is not None:
        o.dt_limit, o.dt_min, o.dt_max = 1, float(dt_limit[0]), float(dt_limit[1])
    if A is None:
        raise ValueError("A is required")
    lead = (ptr["x"], ptr["dt"], _dense(A, "A", _f32, (ch, N), x), ptr["B"], ptr["C"], _dense(D, "D", _f32, (ch,), x))
    return code, lead, _ffi.SelectiveStrides(*st), o, (ch, G, N)


def ssd_selective_forward(x, dt, A, B, C, D=None, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                          dt_limit=None, z=None, want_final=True, stream=None):
    """Selective scan with one dt per channel and one decay per channel and state entry -> (y, final_state or None).

    x, dt, z (batch, L, channels), A (channels, dstate) f32, B, C (batch, L, ngroups, dstate), D (channels,) f32 or
    None, init_state (batch, channels, dstate) f32 or None.  dt <- clamp(softplus(dt + dt_bias), *dt_limit) (each part
    optional) and y <- y * z * sigmoid(z) with a gate."""
    rows = x.shape[:2] if isinstance(x, torch.Tensor) and x.dim() == 3 else (0, 0)
    code, lead, st, o, (ch, G, N) = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, rows)
    b, L = rows
    ip = _dense(init_state, "init_state", _f32, (b, ch, N), x)
    lp = _dense(lengths, "lengths", _i32, (b,), x)
    with _Launch(stream) as s:
        y = x.new_empty((b, L, ch))
        final = x.new_empty((b, ch, N), dtype=_f32) if want_final else None
        _ffi.check("ssd_selective_forward", _ffi.lib().ssd_selective_forward(
            code, *lead, ip, lp, ctypes.addressof(st), b, L, ch, G, N, ctypes.addressof(o), y.data_ptr(),
            None if final is None else final.data_ptr(), s))
    _keep(stream, x, dt, A, B, C, D, init_state, lengths, dt_bias, z)
    return y, final


def ssd_selective_backward(x, dt, A, B, C, D, dy, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                           dt_limit=None, z=None, dfinal=None, want_dinit=False, stream=None):
    """Gradients through ssd_selective_forward given dy (y's layout, dense) and dfinal ((batch, channels, dstate) f32
    or None).

    Returns a dict: dx, ddt (batch, L, channels), dA (channels, dstate) f32, dB, dC (batch, L, ngroups, dstate) f32,
    dD (channels,) f32 or None, ddt_bias (channels,) f32 or None, dz or absent without a gate, dinit (None unless
    wanted)."""
    rows = x.shape[:2] if isinstance(x, torch.Tensor) and x.dim() == 3 else (0, 0)
    code, lead, st, o, (ch, G, N) = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, rows)
    b, L = rows
    ip = _dense(init_state, "init_state", _f32, (b, ch, N), x)
    lp = _dense(lengths, "lengths", _i32, (b,), x)
    if dy is None:
        raise ValueError("dy is required")
    gp = _dense(dy, "dy", x.dtype, (b, L, ch), x)
    fp = _dense(dfinal, "dfinal", _f32, (b, ch, N), x)
    with _Launch(stream) as s:
        out = {"dx": x.new_empty((b, L, ch)), "ddt": x.new_empty((b, L, ch)), "dA": x.new_empty((ch, N), dtype=_f32),
               "dB": x.new_empty((b, L, G, N), dtype=_f32), "dC": x.new_empty((b, L, G, N), dtype=_f32),
               "dD": x.new_empty((ch,), dtype=_f32) if D is not None else None,
               "ddt_bias": x.new_empty((ch,), dtype=_f32) if dt_bias is not None else None,
               "dinit": x.new_empty((b, ch, N), dtype=_f32) if want_dinit else None}
        if z is not None:
            out["dz"] = x.new_empty((b, L, ch))
        p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
        _ffi.check("ssd_selective_backward", _ffi.lib().ssd_selective_backward(
            code, *lead, ip, lp, ctypes.addressof(st), b, L, ch, G, N, ctypes.addressof(o), gp, fp, p["dx"], p["ddt"],
            p["dA"], p["dB"], p["dC"], p["dD"], p.get("dz"), p["ddt_bias"], p["dinit"], s))
    _keep(stream, x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, z, dfinal)
    return out


def ssd_selective_step(x, dt, A, B, C, D, state, slots=None, dt_bias=None, dt_softplus=False, dt_limit=None, z=None,
                       stream=None):
    """ssd_selective_forward for one token of every row -> y (batch, channels).

    x, dt, z (batch, channels), B, C (batch, ngroups, dstate), state (nslots, channels, dstate) f32 updated in place."""
    rows = x.shape[:1] if isinstance(x, torch.Tensor) and x.dim() == 2 else (0,)
    code, lead, st, o, (ch, G, N) = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, rows)
    b = rows[0]
    sp, lp, n = _pool(state, slots, b, (ch, N), _f32, x)
    with _Launch(stream) as s:
        y = x.new_empty((b, ch))
        _ffi.check("ssd_selective_step", _ffi.lib().ssd_selective_step(
            code, *lead, sp, lp, n, ctypes.addressof(st), b, ch, G, N, ctypes.addressof(o), y.data_ptr(), s))
    _keep(stream, x, dt, A, B, C, D, state, slots, dt_bias, z)
    return y


def _flat_rows(t, name, width):
    """(address, row stride, rows) of a tensor whose leading dimensions run through one stride."""
    size, stride = t.shape, t.stride()
    if size[-1] != 1 and stride[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be dense, got strides {stride}")
    step, rows = 0, 1
    for d in range(len(size) - 2, -1, -1):
        if size[d] == 1:
            continue
        if step == 0 and rows == 1:
            step = stride[d]
        elif stride[d] != step * rows:
            raise ValueError(f"the rows of {name} must be evenly spaced, got shape {tuple(size)}, strides {stride}")
        rows *= size[d]
    return t.data_ptr(), step if rows > 1 else width, rows


def ssd_layer_norm_forward(x, weight=None, bias=None, eps=1e-5, stream=None):
    """Layer norm over the last dimension -> (y, mean, rstd).

    x (..., width) with a dense last dimension and evenly spaced rows; weight, bias (width,) f32 or None; y is dense,
    mean and rstd have x's leading shape, f32."""
    code = _dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least 1 dim")
    _input(x, "x", x.dim())
    width = x.shape[-1]
    wp, bp = _dense(weight, "weight", _f32, (width,), x), _dense(bias, "bias", _f32, (width,), x)
    xp, step, rows = _flat_rows(x, "x", width)
    with _Launch(stream) as s:
        y = x.new_empty(x.shape)
        mean, rstd = x.new_empty(x.shape[:-1], dtype=_f32), x.new_empty(x.shape[:-1], dtype=_f32)
        _ffi.check("ssd_layer_norm_forward", _ffi.lib().ssd_layer_norm_forward(
            code, xp, step, wp, bp, float(eps), rows, width, y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), s))
    _keep(stream, x, weight, bias)
    return y, mean, rstd


def ssd_layer_norm_backward(x, weight, mean, rstd, dy, want_dbias=True, stream=None):
    """Gradients through ssd_layer_norm_forward -> dict of dx (dense), dweight (None without a weight) and dbias (None
    unless wanted), both (width,) f32, from the forward pass's mean and rstd."""
    code = _dtype(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least 1 dim")
    _input(x, "x", x.dim())
    width, lead = x.shape[-1], x.shape[:-1]
    wp = _dense(weight, "weight", _f32, (width,), x)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are required")
    mp, rp = _dense(mean, "mean", _f32, lead, x), _dense(rstd, "rstd", _f32, lead, x)
    xp, step, rows = _flat_rows(x, "x", width)
    _check(dy, "dy", x.dtype, x.shape, x)
    gp, gstep, _ = _flat_rows(dy, "dy", width)
    with _Launch(stream) as s:
        out = {"dx": x.new_empty(x.shape), "dweight": x.new_empty((width,), dtype=_f32) if weight is not None else None,
               "dbias": x.new_empty((width,), dtype=_f32) if want_dbias else None}
        p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
        _ffi.check("ssd_layer_norm_backward", _ffi.lib().ssd_layer_norm_backward(
            code, xp, step, wp, mp, rp, gp, gstep, rows, width, p["dx"], p["dweight"], p["dbias"], s))
    _keep(stream, x, weight, mean, rstd, dy)
    return out
