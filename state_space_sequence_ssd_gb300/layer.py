"""The layer operators around a scan: the short causal convolution, the selective scan with one decay per channel
and state entry, the layer norm, the gated linear recurrence, the norm over groups of channels with its gate, and rotary
positions (binding of the ssd_conv_*, ssd_selective_*, ssd_layer_norm_*, ssd_gated_*, ssd_group_norm_* and ssd_rotary
entries of include/ssd.h; the checks of the tensors and the allocation of the outputs are in csrc/layer_binding.cpp).

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


def ssd_gated_forward(x, r, i, A, init_state=None, lengths=None, want_final=True, want_states=False, stream=None):
    """Gated linear recurrence h <- a h + sqrt(1 - a^2) sigmoid(i) x with a = exp(A sigmoid(r)) -> (y, final_state or
    None, states or None).

    x, r, i (batch, L, channels), A (channels,) f32 below zero, init_state (batch, channels) f32 or None; y is the state
    after every token, in x's type.  states (batch, ceil(L / 64), channels) f32 are what ssd_gated_backward takes, the
    state in front of every 64th token."""
    if stream is not None:
        return _on(stream, _native.gated_forward, (x, r, i, A, init_state, lengths, want_final, want_states),
                   (x, r, i, A, init_state, lengths))
    return _native.gated_forward(x, r, i, A, init_state, lengths, want_final, want_states)


def ssd_gated_backward(x, r, i, A, dy, init_state=None, lengths=None, states=None, dfinal=None, want_dinit=False, stream=None):
    """Gradients through ssd_gated_forward given dy (y's layout, dense) and dfinal ((batch, channels) f32 or None) ->
    dict of dx, dr, di (batch, L, channels), dA (channels,) f32, dinit (batch, channels) f32 (None unless wanted).

    states are those of the forward pass on the same inputs (init_state is not read then); None computes them again."""
    if stream is not None:
        return _on(stream, _native.gated_backward, (x, r, i, A, dy, init_state, lengths, states, dfinal, want_dinit),
                   (x, r, i, A, dy, init_state, lengths, states, dfinal))
    return _native.gated_backward(x, r, i, A, dy, init_state, lengths, states, dfinal, want_dinit)


def ssd_gated_step(x, r, i, A, state, slots=None, stream=None):
    """ssd_gated_forward for one token of every row -> y (batch, channels).

    x, r, i (batch, channels); state (nslots, channels) f32 updated in place."""
    if stream is not None:
        return _on(stream, _native.gated_step, (x, r, i, A, state, slots), (x, r, i, A, state, slots))
    return _native.gated_step(x, r, i, A, state, slots)


def ssd_group_norm_forward(x, groups, weight=None, bias=None, z=None, gate_first=False, silu=False, rms=False, eps=1e-5, stream=None):
    """Norm over groups of the last dimension's channels, with its activation -> (y, mean or None, rstd).

    x (..., width) with a dense last dimension and evenly spaced rows, z like it (strides of its own); weight, bias (width,)
    f32 or None; mean (None with ``rms``, which takes it as 0) and rstd are (..., groups) f32.  With a gate z the output is
    norm(x * silu(z)) if ``gate_first``, else norm(x) * silu(z); without one silu(norm(x)) if ``silu``."""
    if stream is not None:
        return _on(stream, _native.group_norm_forward, (x, groups, weight, bias, z, gate_first, silu, rms, eps), (x, weight, bias, z))
    return _native.group_norm_forward(x, groups, weight, bias, z, gate_first, silu, rms, eps)


def ssd_group_norm_backward(x, groups, weight, bias, mean, rstd, dy, z=None, gate_first=False, silu=False, stream=None):
    """Gradients through ssd_group_norm_forward -> dict of dx (dense), dz (absent without a gate), dweight and dbias ((width,)
    f32, None without a weight or a bias), from the forward pass's mean (None: ``rms``) and rstd."""
    if stream is not None:
        return _on(stream, _native.group_norm_backward, (x, groups, weight, bias, mean, rstd, dy, z, gate_first, silu),
                   (x, weight, bias, mean, rstd, dy, z))
    return _native.group_norm_backward(x, groups, weight, bias, mean, rstd, dy, z, gate_first, silu)


def ssd_rotary_table(turned, base=10000.0, scaling=None, factor=1.0, original=None, slow=1.0, fast=32.0, frequencies=None, device="cuda"):
    """The table of the rotary calls for ``turned`` entries of a head -> (turned // 2,) int64 on ``device``: pair k's frequency
    base ** (-2 k / turned) in radians a position, as the part of a turn in units of 2^-64.

    For contexts longer than the ``original`` by ``factor``: scaling "linear" divides every frequency by it, "base" raises the base
    by factor ** (turned / (turned - 2)) (the slowest pair is divided by factor, the fastest kept), "parts" divides those that
    turn less than ``slow`` times over the original context, keeps those that turn more than ``fast`` times, and blends linearly
    between.  ``frequencies`` gives them instead (a sequence of turned // 2 numbers).  The computation is on the host."""
    import math

    import torch
    if turned < 2 or turned % 2:
        raise ValueError(f"turned must be even and at least 2, got {turned}")
    pairs = turned // 2
    if frequencies is None:
        if not base > 0:
            raise ValueError(f"base must be positive, got {base}")
        if not (factor > 0 and math.isfinite(factor)):
            raise ValueError(f"factor must be positive, got {factor}")
        if scaling not in (None, "linear", "base", "parts"):
            raise ValueError(f"scaling must be None, 'linear', 'base' or 'parts', got {scaling!r}")
        if scaling == "base" and turned > 2:
            base = base * factor ** (turned / (turned - 2))
        frequencies = [base ** (-k / pairs) for k in range(pairs)]
        if scaling == "linear" or scaling == "base" and turned == 2:
            frequencies = [f / factor for f in frequencies]
        elif scaling == "parts":
            if original is None or not original > 0 or not fast > slow:
                raise ValueError("scaling 'parts' needs the original context, and fast above slow")
            for k, f in enumerate(frequencies):
                keep = min(max((original * f / (2 * math.pi) - slow) / (fast - slow), 0.0), 1.0)
                frequencies[k] = f * keep + f / factor * (1 - keep)
    else:
        frequencies = [float(f) for f in frequencies]
    if len(frequencies) != pairs or not all(math.isfinite(f) for f in frequencies):
        raise ValueError(f"frequencies must be {pairs} finite numbers")
    turns = [round(f / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for f in frequencies]
    return torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device=device)


def _rotary(args, stream):
    if stream is not None:
        return _on(stream, _native.rotary, args, args[:5])
    return _native.rotary(*args)


def ssd_rotary_forward(B, C, table, positions=None, lengths=None, interleaved=False, scale=1.0, stream=None):
    """Rotary positions on a scan's B and C (or queries and keys) -> (B, C) turned, or B alone where C is None.

    B, C (batch, L, groups, dstate), each with a number of groups of its own; the first 2 * len(table) entries of a group are turned,
    as pairs (2 k, 2 k + 1) if ``interleaved``, else (k, k + len(table)), and multiplied by ``scale``; the others are copied.
    table is ssd_rotary_table's.  Token t is at position t, at positions[b] + t with positions (batch,) int32, or at
    positions[b, t] with (batch, L) int32 (rows of packed documents)."""
    return _rotary((B, C, table, positions, lengths, interleaved, scale, False, False), stream)


def ssd_rotary_backward(dB, dC, table, positions=None, lengths=None, interleaved=False, scale=1.0, stream=None):
    """Gradients through ssd_rotary_forward: (dB, dC) turned back, or dB alone where dC is None."""
    return _rotary((dB, dC, table, positions, lengths, interleaved, scale, True, False), stream)


def ssd_rotary_step(B, C, table, positions, interleaved=False, scale=1.0, stream=None):
    """ssd_rotary_forward for one token of every row: B, C (batch, groups, dstate), positions (batch,) int32."""
    if positions is None:
        raise ValueError("positions is required")
    return _rotary((B, C, table, positions, None, interleaved, scale, False, True), stream)
