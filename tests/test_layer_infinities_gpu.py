"""Live infinities and NaN through the selective scan: what the 64-bit definition makes of them, entry for entry, where dstate
leaves entries, channels and tokens of the kernels' tiles without a use.

Every term is positive (or of one sign per channel), so that the definition's infinities do not meet and their signs are
certain; where it still is NaN the kernels' result has to be NaN or infinite, where it is finite their result has to be close to
it (the tolerances are those of test_layer_gpu.py)."""
import numpy as np
import pytest
import torch

from test_layer_gpu import TYPES, ROUND, Draw, np64, plain_selective, selective_args, spoil, ssd, step_roundings  # noqa: F401

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")

#        type, batch, tokens, channels, groups, dstate, gate, lengths
CASES = [("f32", 2, 40, 8, 1, 3, True, None), ("bf16", 2, 40, 24, 1, 13, True, [40, 37]), ("f16", 2, 50, 12, 2, 1, False, [47, 50]),
         ("f32", 1, 33, 9, 1, 5, True, None), ("bf16", 1, 45, 16, 1, 24, True, [41]), ("f16", 2, 40, 8, 1, 33, False, None),
         ("f32", 2, 60, 8, 2, 100, True, [60, 59]), ("bf16", 2, 40, 32, 1, 16, True, [40, 33]), ("f32", 1, 200, 8, 1, 3, False, None),
         ("bf16", 3, 70, 16, 1, 20, True, [70, 0, 33])]


def case(c, what, seed=17):
    """Inputs of one sign with `what` put into them: (inputs, options, the generator)."""
    kind, b, L, ch, G, N, gate, lengths = c
    d, T = Draw(seed), TYPES[kind]
    some = lambda *shape, dtype=T: (d.normal(*shape).abs() + 0.1).to(dtype)  # noqa: E731
    s = dict(x=some(b, L, ch), A=-torch.exp(d.normal(ch, N, scale=0.3)), dt=d.normal(b, L, ch, dtype=T, scale=0.3), B=some(b, L, G, N),
             C=some(b, L, G, N), D=some(ch, dtype=torch.float32), z=some(b, L, ch) if gate else None,
             bias=d.normal(ch, scale=0.2) - 4, init=some(b, ch, N, dtype=torch.float32),
             lengths=None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    if what == "x":  # two channels, each of one sign
        if ch > 1:
            s["x"][0, L // 3, ch - 1] = -INF
            s["init"][0, ch - 1] *= -1
            s["x"][0, :, ch - 1] *= torch.where(s["x"][0, :, ch - 1] > 0, -1, 1)
        s["x"][0, L // 2, min(1, ch - 1)] = INF
    elif what == "x nan":
        s["x"][0, L // 2, 0] = NAN
    elif what == "dt":
        s["dt"][0, L // 2, min(1, ch - 1)] = INF
    elif what == "last x":  # the row's last token: no later one carries it
        n = L if lengths is None else lengths[0]
        s["x"][0, n - 1, min(1, ch - 1)] = INF
    for k in ("x", "dt", "z", "B", "C"):
        spoil(s[k], s["lengths"], NAN)
    return s, dict(dt_bias=s["bias"], dt_softplus=True, z=s["z"]), d


def agree(name, got, want, mag, roundings):
    rel, least = ROUND[got.dtype]
    g = got.double().cpu().numpy()
    assert g.shape == want.shape, name
    finite = np.isfinite(want)
    tol = rel * np.abs(want[finite]) + least + roundings * 2.0 ** -22 * (1 + rel) * mag[finite]
    bad = ~(np.abs(g[finite] - want[finite]) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} finite ones off, {np.count_nonzero(~np.isfinite(g[finite]))} not finite"
    inf = np.isinf(want)
    assert np.array_equal(g[inf], want[inf]), f"{name}: an infinity became {g[inf][g[inf] != want[inf]][:4]}"
    assert not np.isfinite(g[np.isnan(want)]).any(), f"{name}: a NaN became a number"


def plain(s, opts, **kw):
    """Every row by itself and at its own length: a token past it is not there at all.  (The definition with its magnitudes.)"""
    b, L = s["x"].shape[:2]
    n = [L] * b if s["lengths"] is None else s["lengths"].tolist()
    out = []
    for mag in (False, True):
        rows = []
        for i in range(b):
            cut = {k: v if v is None or k in ("A", "D", "bias", "lengths") else v[i:i + 1] if k == "init" else v[i:i + 1, :n[i]]
                   for k, v in s.items()}
            cut["lengths"] = None
            given = {k: v[i:i + 1] if k == "dfinal" else v[i:i + 1, :n[i]] for k, v in kw.items()}
            with np.errstate(invalid="ignore", over="ignore"):
                rows.append(plain_selective(cut, {"dt_limit": None, **opts, "z": cut["z"]}, mag=mag, **given))
        longer = lambda v, i: np.pad(v, [(0, 0), (0, L - n[i])] + [(0, 0)] * (v.ndim - 2))  # noqa: E731
        if kw:
            summed = ("dA", "dD", "ddt_bias")
            out.append({k: sum(r[k] for r in rows) if k in summed else
                        np.concatenate([r[k] if k == "dinit" else longer(r[k], i) for i, r in enumerate(rows)]) for k in rows[0]})
        else:
            out.append((np.concatenate([longer(r[0], i) for i, r in enumerate(rows)]), np.concatenate([r[1] for r in rows])))
    return out


@pytest.mark.parametrize("what", ["x", "x nan", "dt", "last x"])
@pytest.mark.parametrize("c", CASES)
def test_forward(ssd, c, what):  # noqa: F811
    s, opts, _ = case(c, what)
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], s["lengths"], **opts)
    (ref, rfinal), (mag, mfinal) = plain(s, opts)
    assert what == "x nan" or np.isinf(ref).any()
    k = step_roundings(s) + s["x"].shape[1] + s["A"].shape[1]
    agree("y", y, ref, mag, k + 8)
    agree("final", final, rfinal, mfinal, k)


@pytest.mark.parametrize("what", ["x", "x nan", "dt"])
@pytest.mark.parametrize("c", CASES)
def test_step(ssd, c, what):  # noqa: F811
    """The token that holds the infinity and the one after it, from the state before them."""
    s, opts, _ = case(c[:-1] + (None,), what)
    b, L, ch, G, N = *s["x"].shape, *s["B"].shape[2:]
    state = s["init"].clone()
    for t in (L // 3, L // 2, L // 2 + 1):
        one = {n: v[:, t] if n in ("x", "dt", "B", "C", "z") and v is not None else v for n, v in s.items()}
        row = {n: v[:, t:t + 1] if n in ("x", "dt", "B", "C", "z") and v is not None else v for n, v in s.items()}
        row["init"] = state.clone()
        (ref, rfinal), (mag, mfinal) = plain(row, {**opts, "z": row["z"]})
        y = ssd.ssd_selective_step(*selective_args(one), state, **{**opts, "z": one["z"]})
        k = step_roundings(s) + 1 + N
        agree("y", y, ref[:, 0], mag[:, 0], k + 8)
        agree("state", state, rfinal, mfinal, k)


@pytest.mark.parametrize("what", ["x", "x nan", "dt", "last x", "dy", "B", "C"])
@pytest.mark.parametrize("c", CASES + [("f32", 1, 37, 1, 1, 4, True, None), ("bf16", 1, 44, 2, 2, 16, False, [39])])
def test_backward(ssd, c, what):  # noqa: F811
    """The last two cases have one channel a group, so that the sums over channels have one infinite term."""
    s, opts, d = case(c, what)
    b, L, ch, G, N = *s["x"].shape, *s["B"].shape[2:]
    n = L if c[-1] is None else c[-1][0]
    dy, df = (d.normal(b, L, ch).abs() + 0.1).to(s["x"].dtype), d.normal(b, ch, N).abs() + 0.1
    if what == "dy":
        dy[0, n - 2, ch - 1] = INF
    elif what in ("B", "C"):
        s[what][0, n - 2, G - 1, N - 1] = INF
    spoil(dy, s["lengths"], NAN)
    out = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    ref, mag = plain(s, opts, dy=np64(dy), dfinal=np64(df))
    k = 2 * step_roundings(s) + 2 * L + N + 16
    for name in out:
        if out[name] is not None:
            agree(name, out[name], ref[name], mag[name], k + (ch / 4 if name in ("dB", "dC") else 0 if out[name].dim() > 2 else b * L / 4))


def strong(c, what):
    """Decays of about e^-7 a token: none is zero, but over a chunk or a block of the kernels their product is, in float32."""
    s, opts, d = case(c, what)
    s["A"] = s["A"] - 9
    s["bias"] += 4
    opts["dt_bias"] = s["bias"]
    return s, opts, d


STRONG = [("f32", 1, 200, 8, 1, 16, False, None), ("bf16", 2, 300, 12, 1, 5, True, [300, 150]), ("f16", 1, 130, 8, 2, 20, False, None)]


@pytest.mark.parametrize("what", ["x", "dt", "none"])
@pytest.mark.parametrize("c", STRONG)
def test_forward_carries_an_infinite_state_over_strong_decays(ssd, c, what):  # noqa: F811
    s, opts, _ = strong(c, what)
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], s["lengths"], **opts)
    (ref, rfinal), (mag, mfinal) = plain(s, opts)
    k = step_roundings(s) + s["x"].shape[1] + s["A"].shape[1]
    agree("y", y, ref, mag, k + 8)
    agree("final", final, rfinal, mfinal, k)


@pytest.mark.parametrize("what", ["x", "dy", "none"])
@pytest.mark.parametrize("c", STRONG)
def test_backward_carries_an_infinite_gradient_over_strong_decays(ssd, c, what):  # noqa: F811
    s, opts, d = strong(c, what)
    b, L, ch, N = *s["x"].shape, s["A"].shape[1]
    dy, df = (d.normal(b, L, ch).abs() + 0.1).to(s["x"].dtype), d.normal(b, ch, N).abs() + 0.1
    if what == "dy":
        dy[0, L - 2, ch - 1] = INF
    spoil(dy, s["lengths"], NAN)
    out = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], dfinal=df, want_dinit=True, **opts)
    ref, mag = plain(s, opts, dy=np64(dy), dfinal=np64(df))
    k = 2 * step_roundings(s) + 2 * L + N + 16
    for name in out:
        if out[name] is not None:
            agree(name, out[name], ref[name], mag[name], k + (ch / 4 if name in ("dB", "dC") else 0 if out[name].dim() > 2 else b * L / 4))


@pytest.mark.parametrize("c", [("f32", 2, 40, 8, 1, 3, True, None), ("bf16", 2, 40, 32, 1, 16, True, [40, 33])])
def test_a_nan_dt_is_not_hidden_by_its_limits(ssd, c):  # noqa: F811
    """The channel is NaN from there on, in a prompt, a step and the gradient; the others are as they would be."""
    s, opts, d = case(c, "")
    opts["dt_limit"] = (0.01, 0.03)
    t, ch, N = 20, s["x"].shape[2], s["A"].shape[1]
    s["dt"][0, t, 2] = NAN
    y, final = ssd.ssd_selective_forward(*selective_args(s), s["init"], s["lengths"], **opts)
    (ref, rfinal), (mag, mfinal) = plain(s, opts)
    assert np.isnan(ref[0, t:, 2]).all() and np.isnan(rfinal[0, 2]).all() and np.isfinite(ref[:, :, :2]).all()
    k = step_roundings(s) + s["x"].shape[1] + N
    agree("y", y, ref, mag, k + 8)
    agree("final", final, rfinal, mfinal, k)
    one = {n: v[:, t] if n in ("x", "dt", "B", "C", "z") and v is not None else v for n, v in s.items()}
    step = ssd.ssd_selective_step(*selective_args(one), s["init"].clone(), **{**opts, "z": one["z"]})
    assert bool(torch.isnan(step[0, 2])) and int(torch.isnan(step).sum()) == 1
    dy = (d.normal(*s["x"].shape).abs() + 0.1).to(s["x"].dtype)
    spoil(dy, s["lengths"], NAN)
    out = ssd.ssd_selective_backward(*selective_args(s), dy, s["init"], s["lengths"], **opts)
    ref, mag = plain(s, opts, dy=np64(dy))
    assert np.isnan(ref["dx"][0, t, 2]) and np.isfinite(ref["dx"][1]).all()
    k = 2 * k + s["x"].shape[1] + 16
    for name in ("dx", "ddt", "dz", "dA", "dB", "dC", "dD"):
        agree(name, out[name], ref[name], mag[name], k + (ch / 4 if name in ("dB", "dC") else 0 if out[name].dim() > 2 else 20))
