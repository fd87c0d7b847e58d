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
_empty = torch.empty
_raw_stream = torch._C._cuda_getCurrentRawStream  # the current stream's handle, without a Stream object around it


def _refuse(t, name, dtype, shape, dev):
    """Says what is wrong with a tensor that one of the checks below did not pass."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required" if t is None else f"{name} must be a tensor, got {type(t).__name__}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    raise ValueError(f"{name} must be contiguous")


def _need(t, name, dtype, shape, dev):
    """The address of a dense tensor of this type and shape."""
    if (not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev
            or not t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr()


def _opt(t, name, dtype, shape, dev):
    return None if t is None else _need(t, name, dtype, shape, dev)


def _strides(t, name, inner):
    """The strides of the dimensions before the last `inner`, which have to be dense; 0 for a dimension of one."""
    size, stride = t.shape, t.stride()
    need, n = 1, len(size) - inner
    for d in range(len(size) - 1, n - 1, -1):
        if stride[d] != need and size[d] != 1:
            raise ValueError(f"the last {inner} dimension(s) of {name} must be dense, got strides {stride}")
        need *= size[d]
    if n == 2:
        return (stride[0] if size[0] != 1 else 0), (stride[1] if size[1] != 1 else 0)
    return (stride[0] if size[0] != 1 else 0),


def _rows(t, name, dtype, shape, dev, inner=1):
    """The address and strides of a tensor of rows whose last `inner` dimensions are dense."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dtype, shape, dev)
    return t.data_ptr(), _strides(t, name, inner)


def _input(t, name, ndim):
    """The element type's code, the type and the device of the tensor that leads a call."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} is required")
    T = t.dtype
    code = _TYPES.get(T)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {T}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (no CPU path exists)")
    if ndim and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on {t.device}, which is not the current device")
    return code, T, dev


def _on(stream, call, *inputs):
    """Runs `call` with `stream` as the current one, so that its outputs belong to it, and tells the allocator that
    it uses the inputs."""
    with torch.cuda.stream(stream):
        out = call(None)
    for t in inputs:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def _weights(weight, bias, ch, dev):
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be a (channels, width) tensor")
    W = weight.shape[1]
    return W, _need(weight, "weight", _f32, (ch, W), dev), _opt(bias, "bias", _f32, (ch,), dev)


def _split(splits, channels):
    parts = [channels] if splits is None else [int(n) for n in splits]
    if not 1 <= len(parts) <= 3 or min(parts) < 1 or sum(parts) != channels:
        raise ValueError(f"splits must be one to three positive sizes that add up to {channels}, got {splits}")
    return parts


def _outputs(lead, parts, T, dev):
    """The output's pieces, and their addresses and sizes for the library."""
    if len(parts) == 1:
        y = (_empty((*lead, parts[0]), dtype=T, device=dev),)
        return y, (y[0].data_ptr(), parts[0], None, 0, None, 0)
    y = tuple([_empty((*lead, n), dtype=T, device=dev) for n in parts])
    flat = [v for t, n in zip(y, parts) for v in (t.data_ptr(), n)]
    return y, flat if len(parts) == 3 else (*flat, None, 0)


def ssd_conv_forward(x, weight, bias=None, init_state=None, lengths=None, silu=True, splits=None, want_final=True,
                     stream=None):
    """Short causal depthwise convolution -> (y, final_state or None).

    x (batch, L, channels), weight (channels, width) f32 with width 2 to 4, bias (channels,) f32 or None, init_state
    (batch, width - 1, channels) or None.  y is (batch, L, channels), or with ``splits`` a tuple of dense tensors of
    those numbers of channels (a scan's x, B and C); final_state is the row's last width - 1 inputs."""
    if stream is not None:
        return _on(stream, lambda s: ssd_conv_forward(x, weight, bias, init_state, lengths, silu, splits, want_final, s),
                   x, weight, bias, init_state, lengths)
    code, T, dev = _input(x, "x", 3)
    b, L, ch = x.shape
    W, wp, bp = _weights(weight, bias, ch, dev)
    ip = _opt(init_state, "init_state", T, (b, W - 1, ch), dev)
    lp = _opt(lengths, "lengths", _i32, (b,), dev)
    xb, xt = _strides(x, "x", 1)
    y, flat = _outputs((b, L), _split(splits, ch), T, dev)
    final = _empty((b, W - 1, ch), dtype=T, device=dev) if want_final else None
    status = _ffi.lib().ssd_conv_forward(code, x.data_ptr(), xb, xt, wp, bp, ip, lp, b, L, ch, W, silu, *flat,
                                         final.data_ptr() if want_final else None, _raw_stream(dev))
    if status:
        _ffi.check("ssd_conv_forward", status)
    return (y[0] if splits is None else y), final


def ssd_conv_backward(x, weight, bias, dy, init_state=None, lengths=None, silu=True, dfinal=None, dx=None,
                      want_dinit=False, stream=None):
    """Gradients through ssd_conv_forward -> dict of dx, dweight (channels, width) f32, dbias (channels,) f32 (None
    without a bias), dinit (None unless wanted).

    dy is one tensor or the tuple of pieces, each dense and of x's type or float32; dfinal is the gradient of the
    final state.  ``dx`` may be given: a tensor like x whose last dimension is dense (a slice of a projection's
    gradient)."""
    if stream is not None:
        return _on(stream, lambda s: ssd_conv_backward(x, weight, bias, dy, init_state, lengths, silu, dfinal, dx,
                                                       want_dinit, s),
                   x, weight, bias, *([dy] if isinstance(dy, torch.Tensor) else dy), init_state, lengths, dfinal, dx)
    code, T, dev = _input(x, "x", 3)
    b, L, ch = x.shape
    W, wp, bp = _weights(weight, bias, ch, dev)
    ip = _opt(init_state, "init_state", T, (b, W - 1, ch), dev)
    lp = _opt(lengths, "lengths", _i32, (b,), dev)
    fp = _opt(dfinal, "dfinal", T, (b, W - 1, ch), dev)
    xb, xt = _strides(x, "x", 1)
    pieces = [dy] if isinstance(dy, torch.Tensor) else list(dy)
    parts = _split([p.shape[-1] for p in pieces], ch)
    flat = []
    for i, p in enumerate(pieces):
        wide = p.dtype == _f32
        flat += (_need(p, f"dy[{i}]", _f32 if wide else T, (b, L, parts[i]), dev), parts[i], wide)
    flat += (None, 0, 0) * (3 - len(pieces))
    if dx is None:
        dx = _empty((b, L, ch), dtype=T, device=dev)
    op, (ob, ot) = _rows(dx, "dx", T, (b, L, ch), dev)
    dweight = _empty((ch, W), dtype=_f32, device=dev)
    dbias = _empty((ch,), dtype=_f32, device=dev) if bias is not None else None
    dinit = _empty((b, W - 1, ch), dtype=T, device=dev) if want_dinit else None
    status = _ffi.lib().ssd_conv_backward(
        code, x.data_ptr(), xb, xt, wp, bp, ip, lp, b, L, ch, W, silu, *flat, fp, op, ob, ot, dweight.data_ptr(),
        None if dbias is None else dbias.data_ptr(), None if dinit is None else dinit.data_ptr(), _raw_stream(dev))
    if status:
        _ffi.check("ssd_conv_backward", status)
    return {"dx": dx, "dweight": dweight, "dbias": dbias, "dinit": dinit}


def _pool(state, slots, batch, shape, dtype, dev):
    """The addresses of the states and the slots, and the number of states."""
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError(f"state must be a (slots, {shape[0]}, {shape[1]}) tensor")
    n = state.shape[0]
    if slots is None and n < batch:
        raise ValueError(f"state holds {n} rows for a batch of {batch}")
    return _need(state, "state", dtype, (n, *shape), dev), _opt(slots, "slots", _i32, (batch,), dev), n


def ssd_conv_step(x, weight, bias, state, slots=None, silu=True, splits=None, stream=None):
    """ssd_conv_forward for one token of every row -> y (batch, channels), or the tuple of pieces.

    x (batch, channels); state (nslots, width - 1, channels) of x's type, updated in place."""
    if stream is not None:
        return _on(stream, lambda s: ssd_conv_step(x, weight, bias, state, slots, silu, splits, s), x, weight, bias, state,
                   slots)
    code, T, dev = _input(x, "x", 2)
    b, ch = x.shape
    W, wp, bp = _weights(weight, bias, ch, dev)
    sp, lp, n = _pool(state, slots, b, (W - 1, ch), T, dev)
    xb, = _strides(x, "x", 1)
    y, flat = _outputs((b,), _split(splits, ch), T, dev)
    status = _ffi.lib().ssd_conv_step(code, x.data_ptr(), xb, wp, bp, sp, lp, n, b, ch, W, silu, *flat, _raw_stream(dev))
    if status:
        _ffi.check("ssd_conv_step", status)
    return y[0] if splits is None else y


def _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, ndim):
    """What the three entries share: element type, type, device, the leading arguments, strides, options and sizes."""
    code, T, dev = _input(x, "x", ndim)
    shape = x.shape
    rows, ch = shape[:-1], shape[-1]
    if not isinstance(B, torch.Tensor) or B.dim() != ndim + 1:
        raise ValueError(f"B must be a tensor with {ndim + 1} dims (..., ngroups, dstate)")
    G, N = B.shape[-2:]
    if G < 1 or ch % G:
        raise ValueError(f"ngroups ({G}) must divide channels ({ch})")
    bc = (*rows, G, N)
    xp, xs = x.data_ptr(), _strides(x, "x", 1)
    dp, ds = _rows(dt, "dt", T, shape, dev)
    zp, zs = _rows(z, "z", T, shape, dev) if z is not None else (None, xs)
    Bp, Bs = _rows(B, "B", T, bc, dev, 2)
    Cp, Cs = _rows(C, "C", T, bc, dev, 2)
    if ndim == 3:
        st = _ffi.SelectiveStrides(*xs, *ds, *zs, *Bs, *Cs)
    else:
        st = _ffi.SelectiveStrides(xs[0], 0, ds[0], 0, zs[0], 0, Bs[0], 0, Cs[0], 0)
    bp = _opt(dt_bias, "dt_bias", _f32, (ch,), dev)
    if dt_limit is None:
        o = _ffi.InputOptions(bp, bool(dt_softplus), 0, 0.0, 0.0, 0, zp)
    else:
        o = _ffi.InputOptions(bp, bool(dt_softplus), 1, float(dt_limit[0]), float(dt_limit[1]), 0, zp)
    lead = (code, xp, dp, _need(A, "A", _f32, (ch, N), dev), Bp, Cp, _opt(D, "D", _f32, (ch,), dev))
    return T, dev, lead, st, o, (*rows, ch, G, N)


def ssd_selective_forward(x, dt, A, B, C, D=None, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                          dt_limit=None, z=None, want_final=True, stream=None):
    """Selective scan with one dt per channel and one decay per channel and state entry -> (y, final_state or None).

    x, dt, z (batch, L, channels), A (channels, dstate) f32, B, C (batch, L, ngroups, dstate), D (channels,) f32 or
    None, init_state (batch, channels, dstate) f32 or None.  dt <- clamp(softplus(dt + dt_bias), *dt_limit) (each part
    optional) and y <- y * z * sigmoid(z) with a gate."""
    if stream is not None:
        return _on(stream, lambda s: ssd_selective_forward(x, dt, A, B, C, D, init_state, lengths, dt_bias, dt_softplus,
                                                           dt_limit, z, want_final, s),
                   x, dt, A, B, C, D, init_state, lengths, dt_bias, z)
    T, dev, lead, st, o, sizes = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, 3)
    b, L, ch, _, N = sizes
    ip = _opt(init_state, "init_state", _f32, (b, ch, N), dev)
    lp = _opt(lengths, "lengths", _i32, (b,), dev)
    y = _empty((b, L, ch), dtype=T, device=dev)
    final = _empty((b, ch, N), dtype=_f32, device=dev) if want_final else None
    status = _ffi.lib().ssd_selective_forward(*lead, ip, lp, ctypes.addressof(st), *sizes, ctypes.addressof(o), y.data_ptr(),
                                              final.data_ptr() if want_final else None, _raw_stream(dev))
    if status:
        _ffi.check("ssd_selective_forward", status)
    return y, final


def ssd_selective_backward(x, dt, A, B, C, D, dy, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                           dt_limit=None, z=None, dfinal=None, want_dinit=False, stream=None):
    """Gradients through ssd_selective_forward given dy (y's layout, dense) and dfinal ((batch, channels, dstate) f32
    or None).

    Returns a dict: dx, ddt (batch, L, channels), dA (channels, dstate) f32, dB, dC (batch, L, ngroups, dstate) f32,
    dD (channels,) f32 or None, ddt_bias (channels,) f32 or None, dz (absent without a gate), dinit (None unless
    wanted)."""
    if stream is not None:
        return _on(stream, lambda s: ssd_selective_backward(x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, dt_softplus,
                                                            dt_limit, z, dfinal, want_dinit, s),
                   x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, z, dfinal)
    T, dev, lead, st, o, sizes = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, 3)
    b, L, ch, G, N = sizes
    ip = _opt(init_state, "init_state", _f32, (b, ch, N), dev)
    lp = _opt(lengths, "lengths", _i32, (b,), dev)
    gp = _need(dy, "dy", T, (b, L, ch), dev)
    fp = _opt(dfinal, "dfinal", _f32, (b, ch, N), dev)
    out = {"dx": _empty((b, L, ch), dtype=T, device=dev), "ddt": _empty((b, L, ch), dtype=T, device=dev),
           "dA": _empty((ch, N), dtype=_f32, device=dev), "dB": _empty((b, L, G, N), dtype=_f32, device=dev),
           "dC": _empty((b, L, G, N), dtype=_f32, device=dev),
           "dD": _empty((ch,), dtype=_f32, device=dev) if D is not None else None,
           "ddt_bias": _empty((ch,), dtype=_f32, device=dev) if dt_bias is not None else None,
           "dinit": _empty((b, ch, N), dtype=_f32, device=dev) if want_dinit else None}
    if z is not None:
        out["dz"] = _empty((b, L, ch), dtype=T, device=dev)
    p = {k: None if v is None else v.data_ptr() for k, v in out.items()}
    status = _ffi.lib().ssd_selective_backward(
        *lead, ip, lp, ctypes.addressof(st), *sizes, ctypes.addressof(o), gp, fp, p["dx"], p["ddt"], p["dA"], p["dB"],
        p["dC"], p["dD"], p.get("dz"), p["ddt_bias"], p["dinit"], _raw_stream(dev))
    if status:
        _ffi.check("ssd_selective_backward", status)
    return out


def ssd_selective_step(x, dt, A, B, C, D, state, slots=None, dt_bias=None, dt_softplus=False, dt_limit=None, z=None,
                       stream=None):
    """ssd_selective_forward for one token of every row -> y (batch, channels).

    x, dt, z (batch, channels), B, C (batch, ngroups, dstate), state (nslots, channels, dstate) f32 updated in place."""
    if stream is not None:
        return _on(stream, lambda s: ssd_selective_step(x, dt, A, B, C, D, state, slots, dt_bias, dt_softplus, dt_limit, z,
                                                        s), x, dt, A, B, C, D, state, slots, dt_bias, z)
    T, dev, lead, st, o, (b, ch, G, N) = _selective(x, dt, A, B, C, D, dt_bias, dt_softplus, dt_limit, z, 2)
    sp, lp, n = _pool(state, slots, b, (ch, N), _f32, dev)
    y = _empty((b, ch), dtype=T, device=dev)
    status = _ffi.lib().ssd_selective_step(*lead, sp, lp, n, ctypes.addressof(st), b, ch, G, N, ctypes.addressof(o),
                                           y.data_ptr(), _raw_stream(dev))
    if status:
        _ffi.check("ssd_selective_step", status)
    return y


def _flat_rows(t, name, width):
    """(address, row stride, rows) of a tensor whose leading dimensions run through one stride."""
    size, stride = t.shape, t.stride()
    if stride[-1] != 1 and size[-1] != 1:
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
    if stream is not None:
        return _on(stream, lambda s: ssd_layer_norm_forward(x, weight, bias, eps, s), x, weight, bias)
    code, T, dev = _input(x, "x", 0)
    shape = x.shape
    if not shape:
        raise ValueError("x must have at least 1 dim")
    width = shape[-1]
    wp, bp = _opt(weight, "weight", _f32, (width,), dev), _opt(bias, "bias", _f32, (width,), dev)
    xp, step, rows = _flat_rows(x, "x", width)
    y = _empty(shape, dtype=T, device=dev)
    mean, rstd = _empty(shape[:-1], dtype=_f32, device=dev), _empty(shape[:-1], dtype=_f32, device=dev)
    status = _ffi.lib().ssd_layer_norm_forward(code, xp, step, wp, bp, eps, rows, width, y.data_ptr(), mean.data_ptr(),
                                               rstd.data_ptr(), _raw_stream(dev))
    if status:
        _ffi.check("ssd_layer_norm_forward", status)
    return y, mean, rstd


def ssd_layer_norm_backward(x, weight, mean, rstd, dy, want_dbias=True, stream=None):
    """Gradients through ssd_layer_norm_forward -> dict of dx (dense), dweight (None without a weight) and dbias (None
    unless wanted), both (width,) f32, from the forward pass's mean and rstd."""
    if stream is not None:
        return _on(stream, lambda s: ssd_layer_norm_backward(x, weight, mean, rstd, dy, want_dbias, s), x, weight, mean, rstd,
                   dy)
    code, T, dev = _input(x, "x", 0)
    shape = x.shape
    if not shape:
        raise ValueError("x must have at least 1 dim")
    width, lead = shape[-1], shape[:-1]
    wp = _opt(weight, "weight", _f32, (width,), dev)
    mp, rp = _need(mean, "mean", _f32, lead, dev), _need(rstd, "rstd", _f32, lead, dev)
    xp, step, rows = _flat_rows(x, "x", width)
    if not isinstance(dy, torch.Tensor) or dy.dtype != T or dy.shape != shape or dy.get_device() != dev:
        _refuse(dy, "dy", T, shape, dev)
    gp, gstep, _ = _flat_rows(dy, "dy", width)
    dx = _empty(shape, dtype=T, device=dev)
    dweight = _empty((width,), dtype=_f32, device=dev) if weight is not None else None
    dbias = _empty((width,), dtype=_f32, device=dev) if want_dbias else None
    status = _ffi.lib().ssd_layer_norm_backward(
        code, xp, step, wp, mp, rp, gp, gstep, rows, width, dx.data_ptr(), None if dweight is None else dweight.data_ptr(),
        None if dbias is None else dbias.data_ptr(), _raw_stream(dev))
    if status:
        _ffi.check("ssd_layer_norm_backward", status)
    return {"dx": dx, "dweight": dweight, "dbias": dbias}
