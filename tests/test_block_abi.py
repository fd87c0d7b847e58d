"""The C entries and the binding of the gated recurrence, the grouped norm and the rotary positions refuse bad arguments before they touch a device (no GPU needed)."""
import ctypes
import math

import numpy as np
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


def norm(lib, **kw):
    a = dict(dtype=0, x=FAKE, xr=64, z=None, zr=0, w=FAKE, b=FAKE, eps=1e-5, gate=0, rms=0, rows=4, width=64, groups=8, y=FAKE, mean=FAKE, rstd=FAKE)
    a.update(kw)
    return lib.ssd_group_norm_forward(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(dtype=5), dict(rows=0), dict(width=0), dict(groups=0), dict(groups=5), dict(xr=-1),
                                dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(gate=4), dict(gate=-1), dict(gate=2), dict(gate=3),
                                dict(z=FAKE), dict(z=FAKE, gate=1), dict(z=FAKE, gate=2, zr=-1), dict(z=FAKE + 1, gate=2), dict(w=FAKE + 2),
                                dict(b=FAKE + 1), dict(mean=FAKE + 1), dict(rstd=FAKE + 2), dict(rms=1)])
def test_group_norm_refuses(lib, kw):
    assert norm(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(width=1 << 21, groups=1), dict(width=1 << 17, groups=1 << 17), dict(rows=1 << 41)])
def test_group_norm_unsupported(lib, kw):
    assert norm(lib, **kw) == UNSUPPORTED


def test_group_norm_backward_refuses(lib):
    def call(**kw):
        a = dict(z=FAKE, zr=64, w=FAKE, b=None, gate=3, mean=FAKE, rstd=FAKE, dy=FAKE, dyr=64, rows=4, width=64, groups=8, dx=FAKE, dz=FAKE, dw=FAKE, db=None)
        a.update(kw)
        return lib.ssd_group_norm_backward(0, FAKE, 64, *a.values(), None)
    for kw in (dict(rstd=None), dict(dy=None), dict(dx=None), dict(dz=None), dict(z=None), dict(z=None, gate=0), dict(dyr=-1), dict(rows=0), dict(groups=7),
               dict(dw=FAKE + 1), dict(db=FAKE + 2), dict(dz=FAKE + 1)):
        assert call(**kw) == BAD, kw


def rotary(lib, **kw):
    a = dict(dtype=0, x0=FAKE, b0=4096, t0=64, h0=1, x1=FAKE, b1=4096, t1=64, h1=1, table=FAKE, turned=64, positions=FAKE, each=0, lengths=None, scale=1.0,
             interleaved=0, inverse=0, batch=2, seqlen=64, dim=64, y0=FAKE, y1=FAKE)
    a.update(kw)
    return lib.ssd_rotary(*a.values(), None)


@pytest.mark.parametrize("kw", [dict(x0=None), dict(y0=None), dict(table=None), dict(x1=None), dict(y1=None), dict(h1=0), dict(h0=0), dict(h1=-1), dict(turned=0),
                                dict(turned=63), dict(turned=66), dict(b0=-1), dict(t1=-1), dict(scale=float("nan")), dict(scale=float("inf")),
                                dict(positions=None, each=1), dict(batch=0), dict(seqlen=0), dict(dim=0), dict(dtype=3), dict(table=FAKE + 4), dict(x1=FAKE + 1),
                                dict(positions=FAKE + 2), dict(lengths=FAKE + 1)])
def test_rotary_refuses(lib, kw):
    assert rotary(lib, **kw) == BAD


@pytest.mark.parametrize("kw", [dict(batch=65536), dict(seqlen=1 << 23), dict(h0=1 << 15), dict(h1=1 << 15)])
def test_rotary_unsupported(lib, kw):
    assert rotary(lib, **kw) == UNSUPPORTED


def test_binding_refuses_norms_and_positions_of_the_wrong_kind():
    import state_space_sequence_ssd_gb300 as ssd
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_group_norm_forward(x, 2)
    with pytest.raises(TypeError):
        ssd.ssd_group_norm_forward(x.double(), 2)
    with pytest.raises(ValueError, match="CUDA"):
        ssd.ssd_rotary_forward(torch.zeros((1, 4, 1, 8)), None, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="positions"):
        ssd.ssd_rotary_step(torch.zeros((1, 1, 8)), None, torch.zeros(4, dtype=torch.int64), None)


@pytest.mark.parametrize("kw", [dict(turned=3), dict(turned=0), dict(turned=8, base=0.0), dict(turned=8, scaling="other"), dict(turned=8, factor=0.0),
                                dict(turned=8, scaling="parts", factor=2.0), dict(turned=8, scaling="parts", original=8, slow=2.0, fast=1.0),
                                dict(turned=8, frequencies=[1.0]), dict(turned=4, frequencies=[1.0, float("nan")])])
def test_rotary_table_refuses(kw):
    import state_space_sequence_ssd_gb300 as ssd
    with pytest.raises(ValueError):
        ssd.ssd_rotary_table(device="cpu", **kw)


def test_tables():
    """Long contexts: what each scaling does to the fastest and the slowest pair."""
    import state_space_sequence_ssd_gb300 as m
    turns = lambda **kw: np.array([v % 2 ** 64 for v in m.ssd_rotary_table(64, device="cpu", **kw).tolist()], dtype=np.float64) / 2.0 ** 64 * 2 * math.pi  # noqa: E731
    plain = turns()
    np.testing.assert_allclose(plain, 10000.0 ** (-np.arange(32) / 32), rtol=1e-12)
    np.testing.assert_allclose(turns(scaling="linear", factor=8.0), plain / 8, rtol=1e-12)
    base = turns(scaling="base", factor=8.0)
    np.testing.assert_allclose(base[[0, -1]], [plain[0], plain[-1] / 8], rtol=1e-9)
    parts = turns(scaling="parts", factor=8.0, original=4096)
    rounds = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(parts[rounds > 32], plain[rounds > 32], rtol=1e-12)
    np.testing.assert_allclose(parts[rounds < 1], plain[rounds < 1] / 8, rtol=1e-12)
    assert (np.diff(parts) < 0).all()
