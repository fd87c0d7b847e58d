"""The layer operators around a scan: the short causal convolution, the selective scan with one decay per channel
and state entry, and the layer norm (binding of the ssd_conv_*, ssd_selective_* and ssd_layer_norm_* entries of
include/ssd.h; the checks of the tensors and the allocation of the outputs are in csrc/layer_binding.cpp).

x, dt, z, B, C and the convolution's states are bfloat16, float16 or float32, one type per call; weights, A, D, the
scan's states and every summed gradient are float32.  Inputs may be column slices of a wider tensor: only the last
dimension has to be dense.  ``lengths`` (batch,) int32 says how many tokens of each row count, ``slots`` (batch,)
int32 which state of a pool each row works on (negative: an idle row).  ``stream`` is a torch.cuda.Stream (default:
the current one); outputs are allocated on it.

A tensor of the wrong type raises TypeError, one of the wrong shape, layout or device ValueError, and what the C entry
refuses SSDError.
"""
from __future__ import annotations

import importlib.util
import os

from . import _ffi

_BINDING = os.path.join(os.path.dirname(_ffi.LIB_PATH), "ssd_layer_binding.so")


class _Native:
    """The functions of the binding, which is loaded when one is first asked for (it needs torch and the library)."""

    def __getattr__(self, name):
        if name.startswith("__"):
            raise AttributeError(name)
        if not os.path.exists(_BINDING):
            raise RuntimeError(f"the layer operators' binding was not found at {_BINDING}; build it with "
                               "`python -m state_space_sequence_ssd_gb300.build` (no fallback exists)")
        import torch  # noqa: F401  (its libraries are the binding's)
        _ffi.lib()
        spec = importlib.util.spec_from_file_location("ssd_layer_binding", _BINDING)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.set_fail(_ffi.check)
        self.__dict__.update(vars(module))
        return getattr(module, name)


_native = _Native()


def _on(stream, call, args, inputs):
    """Runs `call` with `stream` as the current one, so that its outputs belong to it, and tells the allocator that
    it uses the inputs."""
    import torch
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in inputs:
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def ssd_conv_forward(x, weight, bias=None, init_state=None, lengths=None, silu=True, splits=None, want_final=True,
                     stream=None):
    """Short causal depthwise convolution -> (y, final_state or None).

    x (batch, L, channels), weight (channels, width) f32 with width 2 to 4, bias (channels,) f32 or None, init_state
    (batch, width - 1, channels) or None.  y is (batch, L, channels), or with ``splits`` a tuple of dense tensors of
    those numbers of channels (a scan's x, B and C); final_state is the row's last width - 1 inputs."""
    if stream is not None:
        return _on(stream, _native.conv_forward, (x, weight, bias, init_state, lengths, silu, splits, want_final),
                   (x, weight, bias, init_state, lengths))
    return _native.conv_forward(x, weight, bias, init_state, lengths, silu, splits, want_final)


def ssd_conv_backward(x, weight, bias, dy, init_state=None, lengths=None, silu=True, dfinal=None, dx=None,
                      want_dinit=False, stream=None):
    """Gradients through ssd_conv_forward -> dict of dx, dweight (channels, width) f32, dbias (channels,) f32 (None
    without a bias), dinit (None unless wanted).

    dy is one tensor or the tuple of pieces, each dense and of x's type or float32; dfinal is the gradient of the
    final state.  ``dx`` may be given: a tensor like x whose last dimension is dense (a slice of a projection's
    gradient)."""
    if stream is not None:
        import torch
        dy = [dy] if isinstance(dy, torch.Tensor) else list(dy)  # an iterator's pieces are taken once
        return _on(stream, _native.conv_backward, (x, weight, bias, dy, init_state, lengths, silu, dfinal, dx, want_dinit),
                   (x, weight, bias, *dy, init_state, lengths, dfinal, dx))
    return _native.conv_backward(x, weight, bias, dy, init_state, lengths, silu, dfinal, dx, want_dinit)


def ssd_conv_step(x, weight, bias, state, slots=None, silu=True, splits=None, stream=None):
    """ssd_conv_forward for one token of every row -> y (batch, channels), or the tuple of pieces.

    x (batch, channels); state (nslots, width - 1, channels) of x's type, updated in place."""
    if stream is not None:
        return _on(stream, _native.conv_step, (x, weight, bias, state, slots, silu, splits),
                   (x, weight, bias, state, slots))
    return _native.conv_step(x, weight, bias, state, slots, silu, splits)


def ssd_selective_forward(x, dt, A, B, C, D=None, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                          dt_limit=None, z=None, want_final=True, stream=None):
    """Selective scan with one dt per channel and one decay per channel and state entry -> (y, final_state or None).

    x, dt, z (batch, L, channels), A (channels, dstate) f32, B, C (batch, L, ngroups, dstate), D (channels,) f32 or
    None, init_state (batch, channels, dstate) f32 or None.  dt <- clamp(softplus(dt + dt_bias), *dt_limit) (each part
    optional) and y <- y * z * sigmoid(z) with a gate."""
    if stream is not None:
        return _on(stream, _native.selective_forward, (x, dt, A, B, C, D, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, want_final),
                   (x, dt, A, B, C, D, init_state, lengths, dt_bias, z))
    return _native.selective_forward(
        x, dt, A, B, C, D, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, want_final)


def ssd_selective_backward(x, dt, A, B, C, D, dy, init_state=None, lengths=None, dt_bias=None, dt_softplus=False,
                           dt_limit=None, z=None, dfinal=None, want_dinit=False, stream=None):
    """Gradients through ssd_selective_forward given dy (y's layout, dense) and dfinal ((batch, channels, dstate) f32
    or None).

    Returns a dict: dx, ddt (batch, L, channels), dA (channels, dstate) f32, dB, dC (batch, L, ngroups, dstate) f32,
    dD (channels,) f32 or None, ddt_bias (channels,) f32 or None, dz (absent without a gate), dinit (None unless
    wanted)."""
    if stream is not None:
        return _on(stream, _native.selective_backward, (x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, dfinal, want_dinit),
                   (x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, z, dfinal))
    return _native.selective_backward(
        x, dt, A, B, C, D, dy, init_state, lengths, dt_bias, dt_softplus, dt_limit, z, dfinal, want_dinit)


def ssd_selective_step(x, dt, A, B, C, D, state, slots=None, dt_bias=None, dt_softplus=False, dt_limit=None, z=None,
                       stream=None):
    """ssd_selective_forward for one token of every row -> y (batch, channels).

    x, dt, z (batch, channels), B, C (batch, ngroups, dstate), state (nslots, channels, dstate) f32 updated in place."""
    if stream is not None:
        return _on(stream, _native.selective_step, (x, dt, A, B, C, D, state, slots, dt_bias, dt_softplus, dt_limit, z),
                   (x, dt, A, B, C, D, state, slots, dt_bias, z))
    return _native.selective_step(x, dt, A, B, C, D, state, slots, dt_bias, dt_softplus, dt_limit, z)


def ssd_layer_norm_forward(x, weight=None, bias=None, eps=1e-5, stream=None):
    """Layer norm over the last dimension -> (y, mean, rstd).

    x (..., width) with a dense last dimension and evenly spaced rows; weight, bias (width,) f32 or None; y is dense,
    mean and rstd have x's leading shape, f32."""
    if stream is not None:
        return _on(stream, _native.norm_forward, (x, weight, bias, eps),
                   (x, weight, bias))
    return _native.norm_forward(x, weight, bias, eps)


def ssd_layer_norm_backward(x, weight, mean, rstd, dy, want_dbias=True, stream=None):
    """Gradients through ssd_layer_norm_forward -> dict of dx (dense), dweight (None without a weight) and dbias (None
    unless wanted), both (width,) f32, from the forward pass's mean and rstd."""
    if stream is not None:
        return _on(stream, _native.norm_backward, (x, weight, mean, rstd, dy, want_dbias),
                   (x, weight, mean, rstd, dy))
    return _native.norm_backward(x, weight, mean, rstd, dy, want_dbias)
