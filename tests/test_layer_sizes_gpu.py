"""GPU parity of the layer operators at the sizes where the launch rules change kernels: long runs of the convolution, several
rows a thread in the steps, wide lanes and long blocks of the selective scan, wide rows of the layer norm in many blocks.
Tolerances and the numbers of roundings are those of test_layer_gpu.py."""
import pytest
import torch

import layer_reference as R
import layer_reference_device as D
from test_layer_gpu import TYPES, ROUND, Draw, close, np64, spoil, ssd, step_roundings  # noqa: F401

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def near(name, got, want, mag, roundings):
    """test_layer_gpu.close, on the device."""
    rel, least = ROUND[got.dtype]
    g = got.double()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    tol = rel * want.abs() + least + roundings * 2.0 ** -22 * (1 + rel) * mag
    bad = ~((g - want).abs() <= tol)
    assert not bool(bad.any()), f"{name}: {int(bad.sum())} of {bad.numel()} off, worst {float(((g - want).abs() / tol).nan_to_num(INF).max()):.3g} of the bound"


def f64(t):
    return None if t is None else t.double() if t.is_floating_point() else t


def i32(v):
    return None if v is None else torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------------------ convolution

#        type, batch, tokens, pieces, width, silu, init, lengths, columns before and after
CONV = [("bf16", 1, 4099, [1024, 128, 128], 4, True, True, [4050], (64, 8)), ("f32", 2, 3700, [333, 308], 3, True, True, [3700, 1234], (1, 0)),
        ("f16", 2, 2500, [1280], 2, False, True, [2500, 65], (0, 0)), ("bf16", 8, 800, [641], 4, True, False, [800, 0, 1, 699, 64, 65, 300, 512], (0, 0))]


def conv_case(c):
    kind, b, L, pieces, W, silu, init, lengths, (before, after) = c
    d, T, ch, n = Draw(41), TYPES[kind], sum(pieces), i32(lengths)
    x = d.wide((b, L), ch, T, before, after)
    spoil(x, n, NAN)
    return d, T, x, d.normal(ch, W, scale=0.5), d.normal(ch), d.normal(b, W - 1, ch, dtype=T) if init else None, n, silu, pieces


@pytest.mark.parametrize("c", CONV)
def test_conv_forward_in_long_runs(ssd, c):  # noqa: F811
    d, T, x, w, bias, init, n, silu, pieces = conv_case(c)
    y, final = ssd.ssd_conv_forward(x, w, bias, init, n, silu=silu, splits=pieces)
    args = [f64(v) for v in (x.nan_to_num(), w, bias, init, n)] + [silu]
    ref, rfinal = D.conv(*args)
    near("y", torch.cat(y, -1), ref, D.conv(*args, mag=True)[0], w.shape[1] + 6)
    assert torch.equal(final.double(), rfinal)


@pytest.mark.parametrize("c", CONV)
def test_conv_backward_in_long_runs(ssd, c):  # noqa: F811
    d, T, x, w, bias, init, n, silu, pieces = conv_case(c)
    b, L, ch = x.shape
    W = w.shape[1]
    dy = [d.normal(b, L, p, dtype=T if i == 0 else torch.float32) for i, p in enumerate(pieces)]
    for v in dy:
        spoil(v, n, NAN)
    df = d.normal(b, W - 1, ch, dtype=T)
    out = ssd.ssd_conv_backward(x, w, bias, dy, init, n, silu=silu, dfinal=df, want_dinit=True)
    args = [f64(v) for v in (x.nan_to_num(), w, bias, init, n)] + [silu]
    kw = dict(dy=torch.cat([v.double() for v in dy], -1).nan_to_num(), dfinal=f64(df))
    ref, mag = D.conv(*args, **kw), D.conv(*args, **kw, mag=True)
    for i, (name, k) in enumerate((("dx", 0), ("dweight", b * L / 4), ("dbias", b * L / 4), ("dinit", 0))):
        near(name, out[name], ref[i], mag[i], 2 * W + 12 + k)


def some_slots(d, batch, pool):
    """Places in the pool, some rows idle, one past the pool; among neighbouring rows too."""
    at = torch.randperm(pool, generator=d.g, device="cuda")[:batch].to(torch.int32)
    at[1::7], at[2::11] = -1, -5
    at[batch - 2] = pool
    return at


@pytest.mark.parametrize("kind,batch,pieces,W,before,after", [("bf16", 66, [8192], 4, 0, 8), ("f16", 77, [900, 101], 3, 1, 3),
                                                              ("f32", 253, [1024, 512], 2, 4, 4), ("f16", 85, [3000, 64, 64], 4, 8, 0)])
def test_conv_step_of_several_rows_a_thread(ssd, kind, batch, pieces, W, before, after):  # noqa: F811
    d, T, ch, pool = Draw(43), TYPES[kind], sum(pieces), batch + 5
    x, w, bias = d.wide((batch,), ch, T, before, after), d.normal(ch, W), d.normal(ch)
    state, at = d.normal(pool, W - 1, ch, dtype=T), some_slots(d, batch, pool)
    was = state.clone()
    y = torch.cat(ssd.ssd_conv_step(x, w, bias, state, at, splits=pieces), -1)
    assert ssd.ssd_get_device_error() == 8
    live = ((at >= 0) & (at < pool)).nonzero()[:, 0]
    slot = at[live].long()
    args = [f64(v) for v in (x[live][:, None], w, bias, was[slot])] + [None, True]
    ref, rfinal = D.conv(*args)
    near("y", y[live], ref[:, 0], D.conv(*args, mag=True)[0][:, 0], W + 6)
    assert torch.equal(state[slot].double(), rfinal)
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[slot] = False
    assert torch.equal(state[rest], was[rest]), "other states are untouched"
    idle = torch.ones(batch, dtype=torch.bool, device="cuda")
    idle[live] = False
    assert int(idle.sum()) > 2 and bool((y[idle] == 0).all())


# ------------------------------------------------------------------------------------------------ selective scan


def selective_case(kind, b, L, ch, G, N, gate=True, lengths=None, around=0, seed=47):
    d, T, n = Draw(seed), TYPES[kind], i32(lengths)
    bc = d.wide((b, L), 2 * G * N, T, around, around)
    s = dict(x=d.normal(b, L, ch, dtype=T), dt=d.normal(b, L, ch, dtype=T), A=-torch.exp(d.normal(ch, N, scale=0.7)),
             B=bc[..., :G * N].unflatten(-1, (G, N)), C=bc[..., G * N:].unflatten(-1, (G, N)), D=d.normal(ch),
             init=d.normal(b, ch, N), lengths=n)
    opts = dict(dt_bias=d.normal(ch, scale=0.5) - 2, dt_softplus=True, z=d.wide((b, L), ch, T, around, around) if gate else None)
    for v in (s["x"], s["dt"], opts["z"], bc):
        spoil(v, n, NAN)
    return d, s, opts


def call(s):
    return [s[k] for k in ("x", "dt", "A", "B", "C", "D")]


def plain(s, opts, **kw):
    args = [f64(v) for v in call(s)] + [f64(s["init"]), s["lengths"]]
    kw = {k: f64(v) for k, v in kw.items()}
    return [D.selective(*args, bias=f64(opts["dt_bias"]), soft=True, z=f64(opts["z"]), mag=m, **kw) for m in (False, True)]


# lanes of four channels and eight entries at 16 entries and fewer: two and one of them a channel, whole and padded, whole
# 16-byte rows and others
@pytest.mark.parametrize("c", [("bf16", 1, 256, 8192, 1, 16), ("f32", 1, 200, 12288, 2, 16, False), ("f16", 2, 256, 8190, 1, 13, True, [256, 201], 1),
                               ("bf16", 4, 256, 4096, 2, 8), ("f16", 2, 256, 8190, 1, 5, False), ("f32", 4, 256, 4096, 2, 8, True, None, 1)])
def test_selective_forward_on_wide_lanes(ssd, c):  # noqa: F811
    d, s, opts = selective_case(*c)
    y, final = ssd.ssd_selective_forward(*call(s), s["init"], s["lengths"], **opts)
    (ref, rfinal), (mag, mfinal) = plain(s, opts)
    k = step_roundings(s) + c[2] + c[5]
    near("y", y, ref, mag, k + 8)
    near("final", final, rfinal, mfinal, k)


@pytest.mark.parametrize("c", [("f16", 2, 256, 8190, 1, 13), ("bf16", 2, 256, 8190, 1, 5, False)])
def test_an_infinity_on_wide_padded_lanes(ssd, c):  # noqa: F811
    """One channel's input is infinite at one token: its outputs are infinities or NaN as the definition's from there on (C and B
    are positive, so that infinities of one sign add up), every other output is as it would be."""
    d, s, opts = selective_case(*c)
    s["B"], s["C"] = s["B"].abs(), s["C"].abs()
    s["x"][0, 100, 4321] = INF
    y, final = ssd.ssd_selective_forward(*call(s), s["init"], **opts)
    (ref, rfinal), (mag, mfinal) = plain(s, opts)
    k = step_roundings(s) + c[2] + c[5]
    for got, want, m in ((y, ref, mag), (final, rfinal, mfinal)):
        f = torch.isfinite(want)
        assert bool((torch.isinf(want).any())) and torch.equal(got.double()[torch.isinf(want)], want[torch.isinf(want)])
        near("finite", got[f], want[f], m[f], k + 8)


# blocks of 32 tokens, several of them, at every number of lanes a channel
@pytest.mark.parametrize("c", [("bf16", 4, 130, 2048, 1, 8), ("f16", 4, 130, 1200, 1, 16, True, [130, 0, 97, 33], 4), ("f32", 3, 100, 1100, 1, 24, False),
                               ("bf16", 2, 130, 640, 2, 64, True, [130, 66]), ("f32", 2, 100, 512, 1, 128, False, None, 1)])
def test_selective_backward_in_long_blocks(ssd, c):  # noqa: F811
    d, s, opts = selective_case(*c)
    b, L, ch = s["x"].shape
    N = s["A"].shape[1]
    dy, df = d.normal(b, L, ch, dtype=s["x"].dtype), d.normal(b, ch, N)
    spoil(dy, s["lengths"], NAN)
    out = ssd.ssd_selective_backward(*call(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    ref, mag = plain(s, opts, dy=dy, dfinal=df)
    k = 2 * step_roundings(s) + 2 * L + N + 16
    more = dict(dA=b * L / 4, dD=b * L / 4, ddt_bias=b * L / 4, dB=ch / 4, dC=ch / 4)
    assert set(out) == set(ref)
    for name in out:
        near(name, out[name], ref[name], mag[name], k + more.get(name, 0))


@pytest.mark.parametrize("kind,batch,ch,G,N,around", [("bf16", 22, 8192, 1, 16, 0), ("f16", 77, 2052, 2, 13, 1), ("f32", 39, 4096, 1, 8, 0),
                                                      ("bf16", 23, 2048, 2, 64, 0), ("f32", 22, 1024, 1, 128, 0), ("bf16", 85, 2048, 1, 24, 8)])
def test_selective_step_of_several_rows_a_thread(ssd, kind, batch, ch, G, N, around):  # noqa: F811
    d, s, opts = selective_case(kind, batch, 1, ch, G, N, around=around)
    pool = batch + 6
    one = {k: v[:, 0] if k in ("x", "dt", "B", "C") else v for k, v in s.items()}
    state, at = d.normal(pool, ch, N), some_slots(d, batch, pool)
    was = state.clone()
    y = ssd.ssd_selective_step(*call(one), state, at, **{**opts, "z": opts["z"][:, 0]})
    assert ssd.ssd_get_device_error() == 8
    live = ((at >= 0) & (at < pool)).nonzero()[:, 0]
    slot = at[live].long()
    cut = {k: v[live] if k in ("x", "dt", "B", "C") else v for k, v in s.items()}
    cut["init"] = was[slot]
    (ref, rfinal), (mag, mfinal) = plain(cut, {**opts, "z": opts["z"][live]})
    k = step_roundings(s) + 1 + N
    near("y", y[live], ref[:, 0], mag[:, 0], k + 8)
    near("state", state[slot], rfinal, mfinal, k)
    rest = torch.ones(pool, dtype=torch.bool, device="cuda")
    rest[slot] = False
    assert torch.equal(state[rest], was[rest]), "other states are untouched"
    idle = torch.ones(batch, dtype=torch.bool, device="cuda")
    idle[live] = False
    assert int(idle.sum()) > 2 and bool((y[idle] == 0).all())


# ------------------------------------------------------------------------------------------------ layer norm


@pytest.mark.parametrize("kind,rows,width,extra", [("bf16", 24, 9000, 0), ("f32", 2600, 4100, 4), ("f16", 41, 4099, 1)])
def test_layer_norm_backward_of_wide_rows_in_many_blocks(ssd, kind, rows, width, extra):  # noqa: F811
    d, T = Draw(53), TYPES[kind]
    x = torch.full((rows, width + extra), NAN, device="cuda", dtype=T)
    x[:, :width] = (d.normal(rows, width) * torch.exp(d.normal(width, scale=0.5)) + 3 * d.normal(rows, 1)).to(T)
    x = x[:, :width]
    w, dy = d.normal(width), d.normal(rows, width, dtype=T)
    _, mean, rstd = ssd.ssd_layer_norm_forward(x, w, None, 1e-5)
    out = ssd.ssd_layer_norm_backward(x, w, mean, rstd, dy)
    ref = R.norm(np64(x), np64(w), None, 1e-5, dy=np64(dy))
    mag = R.norm(np64(x), np64(w), None, 1e-5, dy=np64(dy), mag=True)
    spread = (x.double().abs().mean(-1) * rstd.double()).cpu().numpy()
    close("dx", out["dx"], ref[0], mag[0] * (1 + spread[:, None]), 32)
    close("dweight", out["dweight"], ref[1], mag[1] * (1 + spread.max()), 16 + rows / 4)
    close("dbias", out["dbias"], ref[2], mag[2], 4 + rows / 4)
    again = ssd.ssd_layer_norm_backward(x, w, mean, rstd, dy)
    assert torch.equal(again["dweight"], out["dweight"]) and torch.equal(again["dx"], out["dx"])
