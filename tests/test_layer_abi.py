"""The layer operators' C entries and binding refuse bad arguments before they touch a device (no GPU needed)."""
import ctypes

import pytest
import torch

from state_space_sequence_ssd_gb300 import _ffi, build

FAKE = 4096
BAD, UNSUPPORTED = _ffi.SSD_ERR_INVALID_ARG, _ffi.SSD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return _ffi.lib()


def conv(lib, **kw):
    a = dict(dtype=0, x=FAKE, xb=4096, xt=64, weight=FAKE, bias=FAKE, init=FAKE, lengths=FAKE, batch=2, seqlen=64,
             channels=64, width=4, silu=1, y0=FAKE, n0=64, y1=None, n1=0, y2=None, n2=0, final=FAKE)
    a.update(kw)
    return lib.ssd_conv_forward(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(weight=None), dict(y0=None), dict(dtype=3), dict(dtype=-1), dict(batch=0),
                                dict(seqlen=0), dict(channels=-4), dict(width=0), dict(n0=63), dict(n0=32, n1=32),
                                dict(n0=0, y1=FAKE, n1=64), dict(xb=-1), dict(xt=-8), dict(x=FAKE + 1), dict(bias=FAKE + 2),
                                dict(lengths=FAKE + 2), dict(final=FAKE + 1), dict(n0=128, n1=-64)])
def test_conv_refuses(lib, kw):
    assert conv(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(width=1), dict(width=5), dict(batch=65536), dict(seqlen=1 << 23),
                                dict(channels=1 << 21, n0=1 << 21)])
def test_conv_unsupported(lib, kw):
    assert conv(lib, **kw) == UNSUPPORTED


def conv_backward(lib, **kw):
    a = dict(dtype=0, x=FAKE, xb=4096, xt=64, weight=FAKE, bias=FAKE, init=None, lengths=None, batch=2, seqlen=64, channels=64,
             width=4, silu=1, dy0=FAKE, n0=32, f0=0, dy1=FAKE, n1=32, f1=1, dy2=None, n2=0, f2=0, dfinal=None, dx=FAKE,
             dxb=4096, dxt=64, dw=FAKE, db=FAKE, dinit=None)
    a.update(kw)
    return lib.ssd_conv_backward(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(dx=None), dict(dy1=None), dict(dxt=63), dict(dxt=0), dict(dxb=0), dict(dxb=4095),
                                dict(dy1=FAKE + 2), dict(dw=FAKE + 1), dict(dinit=FAKE + 1), dict(dfinal=FAKE + 1)])
def test_conv_backward_refuses(lib, kw):
    """Among them gradients whose rows would overlap."""
    assert conv_backward(lib, **kw) == BAD


def conv_step(lib, **kw):
    a = dict(dtype=0, x=FAKE, xb=64, weight=FAKE, bias=None, state=FAKE, slots=FAKE, nslots=8, batch=4, channels=64, width=4,
             silu=1, y0=FAKE, n0=64, y1=None, n1=0, y2=None, n2=0)
    a.update(kw)
    return lib.ssd_conv_step(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(state=None), dict(nslots=0), dict(slots=None, nslots=3), dict(slots=FAKE + 1), dict(x=None),
                                dict(batch=0), dict(state=FAKE + 1)])
def test_conv_step_refuses(lib, kw):
    assert conv_step(lib, **kw) == BAD


def selective(lib, options=None, strides=None, **kw):
    a = dict(dtype=2, x=FAKE, dt=FAKE, A=FAKE, B=FAKE, C=FAKE, D=FAKE, init=FAKE, lengths=FAKE)
    n = dict(batch=2, seqlen=64, channels=64, ngroups=2, dstate=16)
    o = dict(y=FAKE, final=FAKE)
    for k, v in kw.items():
        next(d for d in (a, n, o) if k in d)[k] = v
    return lib.ssd_selective_forward(*a.values(), None if strides is None else ctypes.addressof(strides), *n.values(),
                                     None if options is None else ctypes.addressof(options), *o.values(), None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(dt=None), dict(A=None), dict(B=None), dict(C=None), dict(y=None), dict(batch=0),
                                dict(seqlen=-1), dict(channels=0), dict(ngroups=0), dict(ngroups=3), dict(dstate=0), dict(dtype=7),
                                dict(x=FAKE + 2), dict(A=FAKE + 2), dict(final=FAKE + 1), dict(lengths=FAKE + 1), dict(D=FAKE + 3)])
def test_selective_refuses(lib, kw):
    assert selective(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(dstate=129), dict(batch=70000), dict(seqlen=1 << 23), dict(channels=1 << 21)])
def test_selective_unsupported(lib, kw):
    assert selective(lib, **kw) == UNSUPPORTED


def test_selective_refuses_options_and_strides(lib):
    o = _ffi.InputOptions()
    o.dt_limit, o.dt_min, o.dt_max = 1, 0.5, 0.1
    assert selective(lib, options=o) == BAD
    o = _ffi.InputOptions()
    o.z = FAKE + 2
    assert selective(lib, options=o) == BAD
    st = _ffi.SelectiveStrides(*[64] * 9, -1)
    assert selective(lib, strides=st) == BAD


def test_selective_backward_refuses(lib):
    def call(z=None, dz=None, **kw):
        o = _ffi.InputOptions()
        o.z = z
        a = dict(dy=FAKE, dfinal=None, dx=FAKE, ddt=FAKE, dA=FAKE, dB=FAKE, dC=FAKE, dD=None, dz=dz, dbias=None, dinit=None)
        a.update(kw)
        return lib.ssd_selective_backward(2, *[FAKE] * 6, None, None, None, 1, 8, 8, 1, 16, ctypes.addressof(o), *a.values(), None)
    for kw in (dict(dy=None), dict(dx=None), dict(ddt=None), dict(dA=None), dict(dB=None), dict(dC=None), dict(z=FAKE),
               dict(dz=FAKE), dict(dA=FAKE + 2), dict(dx=FAKE + 2)):
        assert call(**kw) == BAD, kw


def test_selective_step_refuses(lib):
    def call(state=FAKE, slots=FAKE, nslots=4, y=FAKE, batch=2, dstate=16):
        return lib.ssd_selective_step(0, *[FAKE] * 6, state, slots, nslots, None, batch, 32, 1, dstate, None, y, None)
    for kw in (dict(state=None), dict(y=None), dict(nslots=0), dict(slots=None, nslots=1), dict(state=FAKE + 2), dict(batch=0)):
        assert call(**kw) == BAD, kw
    assert call(dstate=130) == UNSUPPORTED


def test_layer_norm_refuses(lib):
    def call(dtype=0, x=FAKE, step=64, w=FAKE, b=FAKE, eps=1e-5, rows=4, width=64, y=FAKE, mean=FAKE, rstd=FAKE):
        return lib.ssd_layer_norm_forward(dtype, x, step, w, b, eps, rows, width, y, mean, rstd, None)
    for kw in (dict(x=None), dict(y=None), dict(rows=0), dict(width=0), dict(step=-1), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf")), dict(dtype=9), dict(x=FAKE + 1), dict(mean=FAKE + 2)):
        assert call(**kw) == BAD, kw
    assert call(width=1 << 21) == UNSUPPORTED

    def back(x=FAKE, mean=FAKE, rstd=FAKE, dy=FAKE, dx=FAKE, rows=4, dw=FAKE):
        return lib.ssd_layer_norm_backward(0, x, 64, FAKE, mean, rstd, dy, 64, rows, 64, dx, dw, None, None)
    for kw in (dict(x=None), dict(mean=None), dict(rstd=None), dict(dy=None), dict(dx=None), dict(rows=-1), dict(dw=FAKE + 1)):
        assert back(**kw) == BAD, kw


def test_slot_status_string(lib):
    assert b"SLOT" in lib.ssd_status_string(_ffi.SSD_ERR_SLOT)


def test_binding_refuses_what_is_not_on_the_gpu():
    import state_space_sequence_ssd_gb300 as ssd
    x = torch.zeros((1, 4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_conv_forward(x, torch.zeros((8, 4)))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_layer_norm_forward(x)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_selective_forward(x, x, torch.zeros((8, 4)), x[..., None, :4], x[..., None, :4])
    with pytest.raises(TypeError):
        ssd.ssd_layer_norm_forward(x.double())
    with pytest.raises(ValueError, match="required"):
        ssd.ssd_conv_forward(None, torch.zeros((8, 4)))
    assert "ssd_conv_forward" in ssd.__all__


def test_binding_reads_strides():
    from state_space_sequence_ssd_gb300 import layer
    t = torch.zeros((3, 5, 64))
    assert layer._native.row_strides(t[..., 8:24], 1) == [320, 64]
    assert layer._native.row_strides(t[:1, :, :8], 1) == [0, 64]
    assert layer._native.row_strides(t.unflatten(-1, (4, 16)), 2) == [320, 64]
    with pytest.raises(ValueError, match="dense"):
        layer._native.row_strides(t.transpose(1, 2), 1)
    assert layer._native.flat_rows(t[..., :8]) == (64, 15)
    assert layer._native.flat_rows(t[:1, :1, :8]) == (8, 1)
    with pytest.raises(ValueError, match="evenly"):
        layer._native.flat_rows(t[:, :4])
    with pytest.raises(ValueError, match="required"):
        layer._native.flat_rows(None)
    with pytest.raises(TypeError):
        layer._native.flat_rows(t, t)
