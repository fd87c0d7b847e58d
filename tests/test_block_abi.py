"""The C entries and the binding of the gated recurrence refuse bad arguments before they touch a device (no GPU needed)."""
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


def gated(lib, strides=None, **kw):
    a = dict(dtype=0, x=FAKE, r=FAKE, i=FAKE, A=FAKE, init=None, lengths=None)
    n = dict(batch=2, seqlen=64, channels=64)
    o = dict(y=FAKE, final=None, states=None)
    for k, v in kw.items():
        next(d for d in (a, n, o) if k in d)[k] = v
    return lib.ssd_gated_forward(*a.values(), None if strides is None else ctypes.addressof(strides), *n.values(), *o.values(), None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(r=None), dict(i=None), dict(A=None), dict(y=None), dict(batch=0), dict(seqlen=0),
                                dict(channels=-1), dict(dtype=3), dict(dtype=-1), dict(x=FAKE + 1), dict(r=FAKE + 1), dict(A=FAKE + 2),
                                dict(init=FAKE + 1), dict(lengths=FAKE + 2), dict(final=FAKE + 2), dict(states=FAKE + 1), dict(y=FAKE + 1)])
def test_gated_refuses(lib, kw):
    assert gated(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(batch=65536), dict(seqlen=1 << 23), dict(channels=1 << 21)])
def test_gated_unsupported(lib, kw):
    assert gated(lib, **kw) == UNSUPPORTED


def test_gated_refuses_strides(lib):
    assert gated(lib, strides=_ffi.GatedStrides(64, 64, 64, 64, 64, -1)) == BAD


def test_gated_backward_refuses(lib):
    def call(**kw):
        a = dict(states=None, dy=FAKE, dfinal=None, dx=FAKE, dr=FAKE, di=FAKE, dA=FAKE, dinit=None)
        a.update(kw)
        return lib.ssd_gated_backward(0, *[FAKE] * 4, None, None, None, 1, 8, 8, *a.values(), None)
    for kw in (dict(dy=None), dict(dx=None), dict(dr=None), dict(di=None), dict(dA=None), dict(dA=FAKE + 2), dict(dx=FAKE + 1), dict(dinit=FAKE + 2),
               dict(states=FAKE + 2), dict(dfinal=FAKE + 1)):
        assert call(**kw) == BAD, kw


def test_gated_step_refuses(lib):
    def call(x=FAKE, state=FAKE, slots=FAKE, nslots=4, y=FAKE, batch=2):
        return lib.ssd_gated_step(0, x, FAKE, FAKE, FAKE, state, slots, nslots, None, batch, 32, y, None)
    for kw in (dict(x=None), dict(state=None), dict(y=None), dict(nslots=0), dict(slots=None, nslots=1), dict(state=FAKE + 2), dict(batch=0),
               dict(slots=FAKE + 1)):
        assert call(**kw) == BAD, kw


def test_binding_refuses_what_is_not_on_the_gpu():
    import state_space_sequence_ssd_gb300 as ssd
    x = torch.zeros((1, 4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_gated_forward(x, x, x, torch.zeros(8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_gated_step(x[0], x[0], x[0], torch.zeros(8), torch.zeros((4, 8)))
    with pytest.raises(TypeError):
        ssd.ssd_gated_forward(x.double(), x, x, torch.zeros(8))
    with pytest.raises(ValueError, match="required"):
        ssd.ssd_gated_backward(None, x, x, torch.zeros(8), x)
