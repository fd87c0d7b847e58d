"""The 64-bit definitions that the layer operators' GPU tests compare with, pinned by closed forms, by central
differences and by the framework-independent convolution of torch."""
import numpy as np
import pytest
import torch

import layer_reference as R


def rand(*shape, seed=0, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


@pytest.mark.parametrize("W,silu", [(2, False), (3, True), (4, True)])
def test_conv_matches_torch(W, silu):
    x, w, bias, init = rand(2, 9, 5), rand(5, W, seed=1), rand(5, seed=2), rand(2, W - 1, 5, seed=3)
    y, final = R.conv(x, w, bias, init, None, silu)
    rows = torch.tensor(np.concatenate([init, x], 1))
    want = torch.nn.functional.conv1d(rows.transpose(1, 2), torch.tensor(w)[:, None], torch.tensor(bias), groups=5)
    want = torch.nn.functional.silu(want) if silu else want
    np.testing.assert_allclose(y, want.transpose(1, 2).numpy(), atol=1e-13)
    np.testing.assert_array_equal(final, rows[:, -(W - 1):].numpy())


def test_selective_closed_form_of_a_constant_input():
    """One channel, one entry, constant dt, x = B = C = 1: h_t = dt (1 - a^t) / (1 - a)."""
    L, d, A = 12, 0.3, -0.7
    one = np.ones((1, L, 1))
    y, final = R.selective(one, d * one, np.full((1, 1), A), one[..., None], one[..., None], None, None, None)
    a = np.exp(d * A)
    want = d * (1 - a ** np.arange(1, L + 1)) / (1 - a)
    np.testing.assert_allclose(y[0, :, 0], want, rtol=1e-12)
    np.testing.assert_allclose(final[0, 0, 0], want[-1], rtol=1e-12)


def _directional(f, grads, args, seed):
    """(sum of gradient times direction, central difference of f along it)."""
    rng = np.random.default_rng(seed)
    v = {k: rng.standard_normal(args[k].shape) for k in grads}
    e = 1e-5
    up, down = ({k: args[k] + s * e * v[k] if k in v else args[k] for k in args} for s in (1, -1))
    return sum((grads[k] * v[k]).sum() for k in grads), (f(**up) - f(**down)) / (2 * e)


@pytest.mark.parametrize("lengths", [None, [7, 0, 3]])
@pytest.mark.parametrize("soft,gate", [(True, True), (False, False)])
def test_selective_gradients_against_differences(lengths, soft, gate):
    b, L, ch, G, N = 3, 7, 4, 2, 3
    a = dict(x=rand(b, L, ch), dt=rand(b, L, ch, seed=1) if soft else np.abs(rand(b, L, ch, seed=1)) + 0.01,
             A=-np.abs(rand(ch, N, seed=2)), B=rand(b, L, G, N, seed=3), C=rand(b, L, G, N, seed=4), D=rand(ch, seed=5),
             init=rand(b, ch, N, seed=6), bias=rand(ch, seed=7), z=rand(b, L, ch, seed=8) if gate else None)
    a["bias"] = a["bias"] if soft else np.abs(a["bias"])
    lengths = None if lengths is None else np.array(lengths)
    dy, df = rand(b, L, ch, seed=9), rand(b, ch, N, seed=10)

    def loss(**kw):
        y, final = R.selective(lengths=lengths, soft=soft, **kw)
        return (y * dy).sum() + (final * df).sum()

    g = R.selective(lengths=lengths, soft=soft, dy=dy, dfinal=df, **a)
    names = dict(x="dx", dt="ddt", A="dA", B="dB", C="dC", D="dD", init="dinit", bias="ddt_bias")
    if gate:
        names["z"] = "dz"
    for k, name in names.items():
        got, want = _directional(loss, {k: g[name]}, a, seed=11)
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (name, got, want)


@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients_against_differences(silu):
    b, L, ch, W = 3, 6, 4, 4
    lengths = np.array([6, 0, 2])
    a = dict(x=rand(b, L, ch), w=rand(ch, W, seed=1), bias=rand(ch, seed=2), init=rand(b, W - 1, ch, seed=3))
    dy, df = rand(b, L, ch, seed=4), rand(b, W - 1, ch, seed=5)

    def loss(**kw):
        y, final = R.conv(lengths=lengths, silu=silu, **kw)
        return (y * dy).sum() + (final * df).sum()

    for k, g in zip(("x", "w", "bias", "init"), R.conv(lengths=lengths, silu=silu, dy=dy, dfinal=df, **a)):
        got, want = _directional(loss, {k: g}, a, seed=6)
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (k, got, want)


def test_norm_gradients_against_differences():
    a = dict(x=rand(5, 9) + 3, w=rand(9, seed=1), bias=rand(9, seed=2))
    dy = rand(5, 9, seed=3)

    def loss(**kw):
        return (R.norm(eps=1e-5, **kw)[0] * dy).sum()

    for k, g in zip(("x", "w", "bias"), R.norm(eps=1e-5, dy=dy, **a)):
        got, want = _directional(loss, {k: g}, a, seed=4)
        assert abs(got - want) <= 1e-6 * max(1.0, abs(want)), (k, got, want)
