"""GPU parity of the layer operators (short convolution, selective scan, layer norm) with their 64-bit definitions.

Tolerance.  A float32 evaluation rounds every term of a result a bounded number of times, each by at most 2^-22 of
its magnitude (the approximate exponential and quotient; plain operations 2^-24), so its error is at most
(roundings on the way) * 2^-22 * S, where S is the same sum over the terms' magnitudes (layer_reference, mag=True);
the result is then rounded once to its type, by half its epsilon: 2^-8 (bfloat16, 8 significant bits), 2^-11
(float16; 2^-25 absolute among its subnormals) or 2^-24 (float32).  The number of roundings is written at each test: a fixed number, plus the tokens
that a term is carried over and the terms that are added.
"""
import numpy as np
import pytest
import torch

import layer_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ROUND = {torch.bfloat16: (2.0 ** -8, 0.0), torch.float16: (2.0 ** -11, 2.0 ** -25), torch.float32: (2.0 ** -24, 0.0)}


@pytest.fixture(scope="module")
def ssd():
    from state_space_sequence_ssd_gb300 import build
    build.build()
    import state_space_sequence_ssd_gb300 as m
    m.ssd_get_device_error()
    yield m
    assert m.ssd_get_device_error() == 0


def close(name, got, want, mag, roundings):
    rel, least = ROUND[got.dtype]
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, (name, g.shape, want.shape)
    assert np.isfinite(g).all(), name
    tol = rel * np.abs(want) + least + roundings * 2.0 ** -22 * (1 + rel) * mag
    bad = np.abs(g - want) > tol
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} off, worst {np.max(np.abs(g - want) / np.maximum(tol, 1e-300)):.3g} of the bound"


def np64(t):
    return None if t is None else t.double().cpu().numpy()


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype)

    def wide(self, rows, n, T, before, after):
        """(*rows, n) as a column slice of wider rows; the columns around it are NaN."""
        t = torch.full((*rows, before + n + after), float("nan"), device="cuda", dtype=T)
        t[..., before:before + n] = self.normal(*rows, n, dtype=T)
        return t[..., before:before + n]


def spoil(t, lengths, value):
    """Puts `value` past each row's length."""
    if t is not None and lengths is not None:
        for i, n in enumerate(lengths.tolist()):
            t[i, n:] = value


# ------------------------------------------------------------------------------------------------ convolution

#       type, batch, tokens, pieces, width, silu, bias, init, lengths, columns before and after
CONV = [("bf16", 2, 70, [64], 4, True, True, True, None, (0, 0)),
        ("bf16", 2, 300, [256, 64, 64], 4, True, True, False, None, (256, 4)),
        ("f16", 3, 33, [48, 16, 16], 3, False, False, True, [33, 0, 1], (8, 8)),
        ("f32", 4, 17, [20], 2, True, True, True, [2, 17, 0, 16], (0, 0)),
        ("bf16", 3, 130, [37, 5, 3], 4, True, True, True, [130, 2, 129], (3, 1)),
        ("f16", 1, 1, [8], 4, True, True, True, None, (0, 0)),
        ("f32", 2, 2, [1], 4, False, True, False, None, (5, 2)),
        ("bf16", 1, 5000, [136], 4, True, False, False, None, (0, 0)),
        ("f32", 2, 257, [33, 32], 3, True, True, True, [0, 257], (1, 0))]


def conv_case(c, seed=3):
    kind, b, L, pieces, W, silu, bias, init, lengths, (before, after) = c
    d, T, ch = Draw(seed), TYPES[kind], sum(pieces)
    s = dict(x=d.wide((b, L), ch, T, before, after), weight=d.normal(ch, W, scale=0.5), bias=d.normal(ch) if bias else None,
             init=d.normal(b, W - 1, ch, dtype=T) if init else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    spoil(s["x"], s["lengths"], float("nan"))
    return s, T, pieces, W, silu, d


@pytest.mark.parametrize("c", CONV)
def test_conv_forward(ssd, c):
    s, T, pieces, W, silu, _ = conv_case(c)
    y, final = ssd.ssd_conv_forward(s["x"], s["weight"], s["bias"], s["init"], s["lengths"], silu=silu, splits=pieces)
    n = [np64(s[k]) for k in ("x", "weight", "bias", "init", "lengths")]
    n[0] = np.nan_to_num(n[0])
    ref, rfinal = R.conv(*n, silu)
    mag, _ = R.conv(*n, silu, mag=True)
    assert all(v.is_contiguous() and v.dtype == T for v in y)
    # width + 1 multiply-adds, the sigmoid's exponential and quotient, the product
    close("y", torch.cat(y, -1), ref, mag, W + 6)
    np.testing.assert_array_equal(np64(final), rfinal)
    whole, none = ssd.ssd_conv_forward(s["x"], s["weight"], s["bias"], s["init"], s["lengths"], silu=silu, want_final=False)
    assert none is None and torch.equal(whole, torch.cat(y, -1))


@pytest.mark.parametrize("c", CONV)
@pytest.mark.parametrize("f32_pieces", [False, True])
def test_conv_backward(ssd, c, f32_pieces):
    s, T, pieces, W, silu, d = conv_case(c)
    b, L, ch = s["x"].shape
    dy = tuple(d.normal(b, L, n, dtype=torch.float32 if f32_pieces and i else T) for i, n in enumerate(pieces))
    for v in dy:
        spoil(v, s["lengths"], float("inf"))
    df = d.normal(b, W - 1, ch, dtype=T) if s["init"] is not None else None
    dx = torch.full((b, L, ch + 16), 7.0, device="cuda", dtype=T)  # a slice of a wider gradient
    out = ssd.ssd_conv_backward(s["x"], s["weight"], s["bias"], dy, s["init"], s["lengths"], silu=silu, dfinal=df,
                                dx=dx[..., 8:8 + ch], want_dinit=True)
    n = [np64(s[k]) for k in ("x", "weight", "bias", "init", "lengths")]
    n[0] = np.nan_to_num(n[0])
    gy = np.nan_to_num(np64(torch.cat([v.float() for v in dy], -1)), posinf=0)
    ref = R.conv(*n, silu, dy=gy, dfinal=np64(df))
    mag = R.conv(*n, silu, dy=gy, dfinal=np64(df), mag=True)
    # pre's W + 1 roundings, the slope's eight, the W + 1 terms; the weights' sums add up to batch * tokens terms
    k = 2 * W + 12
    close("dx", out["dx"], ref[0], mag[0], k)
    close("dweight", out["dweight"], ref[1], mag[1], k + b * L / 4)
    if s["bias"] is not None:
        close("dbias", out["dbias"], ref[2], mag[2], k + b * L / 4)
    else:
        assert out["dbias"] is None
    close("dinit", out["dinit"], ref[3], mag[3], k)
    assert out["dx"].data_ptr() == dx[..., 8:].data_ptr()
    assert bool((dx[..., :8] == 7).all()) and bool((dx[..., 8 + ch:] == 7).all()), "the columns around dx are untouched"
    again = ssd.ssd_conv_backward(s["x"], s["weight"], s["bias"], dy, s["init"], s["lengths"], silu=silu, dfinal=df)
    assert torch.equal(again["dweight"], out["dweight"]) and torch.equal(again["dx"], out["dx"])


def test_conv_narrow_taps_ignore_older_tokens(ssd):
    """A width of 2 reads no third token, whatever it holds."""
    x = torch.zeros((1, 8, 16), device="cuda")
    x[0, 2] = float("inf")
    y, _ = ssd.ssd_conv_forward(x, torch.ones((16, 2), device="cuda"), silu=False)
    assert bool(torch.isinf(y[0, 2:4]).all()) and bool((y[0, 4:] == 0).all())


@pytest.mark.parametrize("kind,ch,W,before", [("bf16", 64, 4, 0), ("f16", 50, 3, 1), ("f32", 33, 2, 4), ("bf16", 384, 4, 256)])
def test_conv_steps_continue_the_prompt(ssd, kind, ch, W, before):
    """A prompt, then single tokens from its final state in slots of a pool: the outputs of one longer prompt."""
    d, T, b, L, more = Draw(5), TYPES[kind], 3, 11, 4
    x, w, bias = d.wide((b, L + more), ch, T, before, 3), d.normal(ch, W), d.normal(ch)
    want, wfinal = ssd.ssd_conv_forward(x, w, bias)
    y, final = ssd.ssd_conv_forward(x[:, :L], w, bias)
    assert torch.equal(y, want[:, :L])
    pool = torch.full((7, W - 1, ch), 9.0, device="cuda", dtype=T)
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = final
    for t in range(more):
        got = ssd.ssd_conv_step(x[:, L + t], w, bias, pool, slots)
        assert torch.equal(got, want[:, L + t])
    assert torch.equal(pool[slots.long()], wfinal)
    assert bool((pool[[1, 2, 3, 5]] == 9).all()), "other states are untouched"


# ------------------------------------------------------------------------------------------------ selective scan

#       type, batch, tokens, channels, groups, dstate, softplus, gate, D, init, lengths, limit, columns around z / B, C
SEL = [("bf16", 2, 40, 32, 1, 16, True, True, True, True, None, None, 0),
       ("f32", 1, 1, 8, 1, 16, True, True, True, True, None, None, 0),
       ("f32", 2, 65, 33, 1, 13, True, False, True, False, None, None, 1),
       ("f16", 4, 129, 60, 2, 8, True, True, False, True, [129, 0, 1, 64], None, 4),
       ("f32", 3, 64, 6, 3, 1, False, True, True, True, [0, 63, 64], None, 0),
       ("bf16", 2, 100, 24, 2, 33, True, True, True, True, [99, 33], (0.01, 0.3), 3),
       ("f32", 1, 70, 9, 1, 64, True, True, True, True, None, (0.02, 0.5), 0),
       ("f16", 2, 31, 4, 1, 128, True, False, True, True, [31, 8], None, 8),
       ("f32", 2, 1300, 20, 1, 16, True, True, True, True, [1300, 777], None, 0),
       ("bf16", 1, 2050, 8, 1, 5, True, True, True, True, None, None, 2),
       ("f32", 1, 3, 1, 1, 2, False, False, False, False, None, None, 0),
       ("bf16", 1, 16, 260, 4, 17, True, True, True, False, None, None, 0),
       ("f16", 2, 77, 534, 2, 13, True, True, True, True, [77, 30], None, 1), ("bf16", 3, 45, 7, 1, 3, True, True, True, False, None, None, 1),
       ("bf16", 1, 66, 129, 3, 9, True, False, True, True, None, None, 3), ("f16", 2, 50, 535, 1, 20, True, True, False, True, [50, 49], None, 1),
       ("bf16", 2, 40, 31, 1, 27, True, False, True, True, None, None, 2), ("f32", 2, 90, 135, 1, 19, True, True, True, True, None, None, 1),
       ("bf16", 4, 130, 1200, 1, 16, True, True, True, True, None, None, 0), ("f16", 4, 130, 1201, 1, 13, True, False, True, True, [130, 0, 95, 64], None, 1),
       ("f32", 1, 24, 40, 1, 16, True, True, True, True, None, None, 0), ("f32", 2, 16, 12, 1, 40, True, True, True, True, [16, 0], None, 0)]


def selective_case(c, seed=7):
    kind, b, L, ch, G, N, soft, gate, D, init, lengths, limit, around = c
    d, T = Draw(seed), TYPES[kind]
    bc = d.wide((b, L), 2 * G * N, T, around, around)
    s = dict(x=d.normal(b, L, ch, dtype=T), A=-torch.exp(d.normal(ch, N, scale=0.7)),
             dt=d.normal(b, L, ch, dtype=T) if soft else (0.2 * d.normal(b, L, ch).abs()).to(T),
             B=bc[..., :G * N].unflatten(-1, (G, N)), C=bc[..., G * N:].unflatten(-1, (G, N)), D=d.normal(ch) if D else None,
             z=d.wide((b, L), ch, T, around, around) if gate else None, bias=d.normal(ch, scale=0.5) - 2 if soft else None,
             init=d.normal(b, ch, N) if init else None,
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    for k in ("x", "dt", "z"):
        spoil(s[k], s["lengths"], float("nan"))
    spoil(bc, s["lengths"], float("inf"))
    return s, T, dict(dt_bias=s["bias"], dt_softplus=soft, dt_limit=limit, z=s["z"]), d


def plain_selective(s, opts, **kw):
    lengths = None if s["lengths"] is None else s["lengths"].cpu().numpy()
    return R.selective(np64(s["x"]), np64(s["dt"]), np64(s["A"]), np64(s["B"]), np64(s["C"]), np64(s["D"]), np64(s["init"]),
                       lengths, bias=np64(s["bias"]), soft=opts["dt_softplus"], limit=opts["dt_limit"], z=np64(s["z"]), **kw)


def selective_args(s):
    return [s[k] for k in ("x", "dt", "A", "B", "C", "D")]


def step_roundings(s):
    """Roundings of one token's decay in units of 2^-22: exp(v) of a rounded v is off by |v| roundings."""
    return 8 + 4 * float(s["A"].abs().max())


@pytest.mark.parametrize("c", SEL)
def test_selective_forward(ssd, c):
    s, T, opts, _ = selective_case(c)
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], s["lengths"], **opts)
    with np.errstate(invalid="ignore"):
        ref, rfinal = plain_selective(s, opts)
        mag, mfinal = plain_selective(s, opts, mag=True)
    L, N = s["x"].shape[1], s["A"].shape[1]
    k = step_roundings(s) + L + N
    close("y", y, ref, mag, k + 8)
    close("final", final, rfinal, mfinal, k)
    y2, none = ssd.ssd_selective_forward(*selective_args(s), s["init"], s["lengths"], want_final=False, **opts)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("c", SEL)
def test_selective_backward(ssd, c):
    s, T, opts, d = selective_case(c)
    b, L, ch = s["x"].shape
    N = s["A"].shape[1]
    dy, df = d.normal(b, L, ch, dtype=T), d.normal(b, ch, N) if s["init"] is not None else None
    spoil(dy, s["lengths"], float("nan"))
    out = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    with np.errstate(invalid="ignore"):
        ref = plain_selective(s, opts, dy=np64(dy), dfinal=np64(df))
        mag = plain_selective(s, opts, dy=np64(dy), dfinal=np64(df), mag=True)
    # a term is carried by a state and by its gradient: up to L tokens in all, each way
    k = 2 * step_roundings(s) + 2 * L + N + 16
    for name in ("dx", "ddt", "dz", "dinit"):
        if name == "dz" and s["z"] is None:
            assert "dz" not in out
        else:
            close(name, out[name], ref[name], mag[name], k)
    close("dA", out["dA"], ref["dA"], mag["dA"], k + b * L / 4)
    for name in ("dB", "dC"):
        close(name, out[name], ref[name], mag[name], k + ch / 4)
    for name, t in (("dD", s["D"]), ("ddt_bias", s["bias"])):
        if t is None:
            assert out[name] is None
        else:
            close(name, out[name], ref[name], mag[name], k + b * L / 4)
    again = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    assert all(v is None or torch.equal(v, again[name]) for name, v in out.items()), "two calls differ"


def test_selective_gradients_against_differences(ssd):
    """The kernel's gradients times a direction, and the difference of the 64-bit loss along it."""
    s, T, opts, d = selective_case(("f32", 2, 37, 12, 2, 5, True, True, True, True, [37, 20], None, 0))
    s["x"], s["dt"], s["z"], s["B"], s["C"] = (torch.nan_to_num(s[k], posinf=0.0).contiguous() for k in ("x", "dt", "z", "B", "C"))
    opts["z"] = s["z"]
    dy, df = d.normal(2, 37, 12), d.normal(2, 12, 5)
    out = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", bias="ddt_bias", z="dz", init="dinit")
    for k, name in names.items():
        v = d.normal(*s[k].shape)
        loss = []
        for sign in (1, -1):
            t = {**s, k: s[k].double() + sign * 1e-4 * v.double()}
            y, final = plain_selective(t, {**opts, "z": t["z"]})
            loss.append((y * np64(dy)).sum() + (final * np64(df)).sum())
        want = (loss[0] - loss[1]) / 2e-4
        got = float((out[name].double() * v.double()).sum())
        scale = float((out[name].double() * v.double()).abs().sum())
        # the difference's own error (second order in 1e-4, third derivatives of order one) and float32 sums
        assert abs(got - want) <= 1e-5 * scale + 1e-5, (name, got, want)


@pytest.mark.parametrize("kind,ch,G,N", [("f32", 40, 1, 16), ("bf16", 36, 2, 13), ("f16", 8, 1, 64), ("f32", 7, 1, 128)])
def test_selective_steps_continue_the_prompt(ssd, kind, ch, G, N):
    """A prompt in two calls, the second one token by token on slots of a pool, against one 64-bit run."""
    L, more, b = 50, 5, 3
    s, T, opts, d = selective_case((kind, b, L + more, ch, G, N, True, True, True, True, None, None, 2))
    ref, rfinal = plain_selective(s, opts)
    mag, mfinal = plain_selective(s, opts, mag=True)
    cut = {k: (v[:, :L] if k in ("x", "dt", "B", "C", "z") else v) for k, v in s.items()}
    y, final = ssd.ssd_selective_forward(*selective_args(cut), s["init"], **{**opts, "z": cut["z"]})
    k = step_roundings(s) + L + more + N + 8
    close("y", y, ref[:, :L], mag[:, :L], k)
    pool = torch.full((9, ch, N), 3.0, device="cuda")
    slots = torch.tensor([8, 2, 5], dtype=torch.int32, device="cuda")
    pool[slots.long()] = final
    for t in range(L, L + more):
        one = {n: (v[:, t] if n in ("x", "dt", "B", "C", "z") else v) for n, v in s.items()}
        got = ssd.ssd_selective_step(*selective_args(one), pool, slots, **{**opts, "z": one["z"]})
        close("step", got, ref[:, t], mag[:, t], k)
    close("state", pool[slots.long()], rfinal, mfinal, k)
    assert bool((pool[[0, 1, 3, 4, 6, 7]] == 3).all())


def test_selective_split_prompts_agree(ssd):
    """One call against two that hand the state over, at a length that is split into chunks on its own."""
    s, T, opts, _ = selective_case(("f32", 1, 3000, 16, 1, 16, True, True, True, True, None, None, 0))
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], **opts)
    parts, state = [], s["init"]
    for a, e in ((0, 1111), (1111, 3000)):
        cut = {k: (v[:, a:e] if k in ("x", "dt", "B", "C", "z") else v) for k, v in s.items()}
        yy, state = ssd.ssd_selective_forward(*selective_args(cut), state, **{**opts, "z": cut["z"]})
        parts.append(yy)
    mag, mfinal = plain_selective(s, opts, mag=True)
    k = 2 * (step_roundings(s) + 3000 + 16)
    close("y", y, np64(torch.cat(parts, 1)), mag, k)
    close("final", final, np64(state), mfinal, k)


# ------------------------------------------------------------------------------------------------ steps: idle rows

@pytest.mark.parametrize("op", ["conv", "selective"])
def test_idle_and_wrong_slots(ssd, op):
    b, ch, n = 5, 24, 6
    d = Draw(2)
    slots = torch.tensor([3, -1, 0, -7, 6], dtype=torch.int32, device="cuda")  # the last is past the pool
    x = d.normal(b, ch)
    x[1], x[3] = float("nan"), float("nan")  # what an idle row holds is not used
    if op == "conv":
        state = d.normal(n, 3, ch)
        before = state.clone()
        y = ssd.ssd_conv_step(x, d.normal(ch, 4), None, state, slots)
    else:
        state = d.normal(n, ch, 8)
        before = state.clone()
        y = ssd.ssd_selective_step(x, x.abs(), -d.normal(ch, 8).abs(), d.normal(b, 1, 8), d.normal(b, 1, 8), None, state, slots)
    assert ssd.ssd_get_device_error() == 8
    assert ssd.ssd_get_device_error() == 0, "reading the error clears it"
    assert bool((y[[1, 3, 4]] == 0).all()) and bool(torch.isfinite(y).all()) and bool((y[[0, 2]] != 0).any())
    assert torch.equal(state[[1, 2, 4, 5]], before[[1, 2, 4, 5]])
    assert not torch.equal(state[3], before[3]) and not torch.equal(state[0], before[0])


# ------------------------------------------------------------------------------------------------ layer norm

NORM = [("bf16", 5, 64, 0), ("f16", 3, 1, 0), ("f32", 300, 7, 0), ("bf16", 1, 2048, 0), ("f32", 2, 31, 1), ("f16", 33, 1000, 8),
        ("bf16", 9, 2049, 0), ("f32", 17, 1024, 4), ("bf16", 4, 16384, 0), ("f16", 2, 20000, 0), ("f32", 3, 9001, 2),
        ("bf16", 700, 512, 0), ("f32", 1000, 24, 0), ("bf16", 5001, 1000, 0), ("f16", 20001, 49, 0), ("f32", 9999, 260, 4),
        ("f32", 4001, 1028, 4), ("bf16", 60001, 64, 0), ("f16", 500, 8000, 8)]


def norm_case(c, seed=13):
    kind, rows, width, extra = c
    d, T = Draw(seed), TYPES[kind]
    x = torch.full((rows, width + extra), float("nan"), device="cuda", dtype=T)
    x[:, :width] = (d.normal(rows, width) * torch.exp(d.normal(width, scale=0.5)) + 3 * d.normal(rows, 1)).to(T)
    return x[:, :width], T, d


@pytest.mark.parametrize("c", NORM)
@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm(ssd, c, affine):
    x, T, d = norm_case(c)
    rows, width = x.shape
    w, bias = (d.normal(width), d.normal(width)) if affine else (None, None)
    y, mean, rstd = ssd.ssd_layer_norm_forward(x, w, bias, 1e-5)
    ref, rmean, rrstd = R.norm(np64(x), np64(w), np64(bias), 1e-5)
    mag = R.norm(np64(x), np64(w), np64(bias), 1e-5, mag=True)[0]
    close("mean", mean, rmean, np.abs(np64(x)).mean(-1), 8)
    # a sum's error grows with the logarithm of its length and a thread's own columns; the variance's error moves
    # rstd by half of it, and the mean's error (relative to the magnitudes) moves every entry
    spread = np.abs(np64(x)).mean(-1) * rrstd
    close("rstd", rstd, rrstd, rrstd * (1 + spread), 12)
    close("y", y, ref, mag * (1 + spread[:, None]), 16)
    dy = d.normal(rows, width, dtype=T)
    out = ssd.ssd_layer_norm_backward(x, w, mean, rstd, dy, want_dbias=affine)
    gref = R.norm(np64(x), np64(w), None, 1e-5, dy=np64(dy))
    gmag = R.norm(np64(x), np64(w), None, 1e-5, dy=np64(dy), mag=True)
    worst = 1 + spread.max()
    close("dx", out["dx"], gref[0], gmag[0] * (1 + spread[:, None]), 32)
    if affine:
        close("dweight", out["dweight"], gref[1], gmag[1] * worst, 16 + rows / 4)
        close("dbias", out["dbias"], gref[2], gmag[2], 4 + rows / 4)
        again = ssd.ssd_layer_norm_backward(x, w, mean, rstd, dy)
        assert torch.equal(again["dweight"], out["dweight"]) and torch.equal(again["dx"], out["dx"])
    else:
        assert out["dweight"] is None and out["dbias"] is None


def test_layer_norm_of_constant_rows(ssd):
    """No spread: y is the bias, rstd 1 / sqrt(eps)."""
    x = torch.full((3, 40), 5.0, device="cuda")
    bias = torch.arange(40, device="cuda").float()
    y, mean, rstd = ssd.ssd_layer_norm_forward(x, None, bias, 0.25)
    assert torch.equal(y, bias.expand(3, 40)) and bool((mean == 5).all()) and bool((rstd == 2).all())


def test_layer_norm_takes_leading_dimensions(ssd):
    d = Draw(1)
    x = d.normal(4, 6, 3 * 32)[..., 32:64]
    y, mean, rstd = ssd.ssd_layer_norm_forward(x)
    y2, _, _ = ssd.ssd_layer_norm_forward(x.reshape(24, 32).contiguous())
    assert y.shape == (4, 6, 32) and mean.shape == rstd.shape == (4, 6) and torch.equal(y.reshape(24, 32), y2)


# ------------------------------------------------------------------------------------------------ streams

def test_another_stream(ssd):
    """Inputs made on one stream, used on another: the results are those of the first."""
    s, T, opts, d = selective_case(("f32", 2, 400, 24, 1, 16, True, True, True, True, None, None, 0))
    want, wfinal = ssd.ssd_selective_forward(*selective_args(s), s["init"], **opts)
    w = d.normal(24, 4)
    cy, _ = ssd.ssd_conv_forward(s["x"], w)
    ny, _, _ = ssd.ssd_layer_norm_forward(s["x"])
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], stream=other, **opts)
    cy2, _ = ssd.ssd_conv_forward(s["x"], w, stream=other)
    ny2, _, _ = ssd.ssd_layer_norm_forward(s["x"], stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(y, want) and torch.equal(final, wfinal) and torch.equal(cy, cy2) and torch.equal(ny, ny2)


# ------------------------------------------------------------------------------------------------ long strides

def test_offsets_past_32_bits(ssd):
    """Slices of rows so wide that the last tokens lie more than 2^31 elements on: the results are those of dense copies."""
    d, T, L, ch, N = Draw(4), torch.bfloat16, 2200, 40, 8
    wide = torch.empty(1, L, 1 << 20, device="cuda", dtype=T)
    assert wide.stride(1) * (L - 1) > 2 ** 31
    wide[..., :4 * ch + 2 * N] = d.normal(1, L, 4 * ch + 2 * N, dtype=T)
    x, dt, z, dx = (wide[..., i * ch:(i + 1) * ch] for i in range(4))
    B, C = (wide[..., 4 * ch + i * N:4 * ch + (i + 1) * N].unflatten(-1, (1, N)) for i in range(2))
    dense = lambda *ts: [t.contiguous() for t in ts]
    w, bias, A, dy = d.normal(ch, 4), d.normal(ch), -d.normal(ch, N).abs(), d.normal(1, L, ch, dtype=T)

    def same(a, b):
        a, b = ([v for v in (o.values() if isinstance(o, dict) else o) if v is not None] for o in (a, b))
        assert len(a) == len(b) and all(torch.equal(p, q) for p, q in zip(a, b))

    same(ssd.ssd_conv_forward(x, w, bias), ssd.ssd_conv_forward(*dense(x), w, bias))
    want = ssd.ssd_conv_backward(*dense(x), w, bias, dy)
    same(ssd.ssd_conv_backward(x, w, bias, dy, dx=dx), want)
    assert torch.equal(dx, want["dx"])
    opts = dict(dt_bias=bias, dt_softplus=True)
    same(ssd.ssd_selective_forward(x, dt, A, B, C, bias, z=z, **opts),
         ssd.ssd_selective_forward(*dense(x, dt), A, *dense(B, C), bias, z=z.contiguous(), **opts))
    same(ssd.ssd_selective_backward(x, dt, A, B, C, bias, dy, z=z, **opts),
         ssd.ssd_selective_backward(*dense(x, dt), A, *dense(B, C), bias, dy, z=z.contiguous(), **opts))
    want = ssd.ssd_layer_norm_forward(*dense(x[0]), w[:, 0].contiguous(), bias)
    same(ssd.ssd_layer_norm_forward(x[0], w[:, 0].contiguous(), bias), want)
    same(ssd.ssd_layer_norm_backward(x[0], w[:, 0].contiguous(), *want[1:], dy[0]),
         ssd.ssd_layer_norm_backward(*dense(x[0]), w[:, 0].contiguous(), *want[1:], dy[0]))


@pytest.mark.parametrize("op", ["conv", "selective"])
def test_slots_past_32_bits(ssd, op):
    """A pool whose last slots lie more than 2^31 elements on."""
    d, ch = Draw(6), 512
    rest = (4, ch) if op == "selective" else (3, ch)
    n = 2 ** 31 // (rest[0] * ch) + 3
    pool = torch.empty(n, *((ch, 4) if op == "selective" else rest), device="cuda", dtype=torch.float32)
    slots = torch.tensor([n - 1, 1, n - 2], dtype=torch.int32, device="cuda")
    small = d.normal(3, *pool.shape[1:])
    pool[slots.long()] = small
    x = d.normal(3, ch)
    if op == "conv":
        run = lambda state, at: ssd.ssd_conv_step(x, w, None, state, at)
        w = d.normal(ch, 4)
    else:
        run = lambda state, at: ssd.ssd_selective_step(x, x.abs(), A, B, B, None, state, at)
        A, B = -d.normal(ch, 4).abs(), d.normal(3, 1, 4)
    y = run(pool, slots)
    assert torch.equal(y, run(small, None)) and torch.equal(pool[slots.long()], small)
