"""The 64-bit definitions on torch tensors that test_layer_sizes_gpu.py compares with are those of layer_reference (no GPU
needed)."""
import numpy as np
import pytest
import torch

import layer_reference as R
import layer_reference_device as D


def rand(*shape, seed, scale=1.0):
    return np.random.default_rng(seed).standard_normal(shape) * scale


def both(plain, device, args, kw):
    as_torch = lambda v: torch.tensor(v) if isinstance(v, np.ndarray) else v  # noqa: E731
    got = device(*map(as_torch, args), **{k: as_torch(v) for k, v in kw.items()})
    want = plain(*args, **kw)
    pairs = [(got[k], want[k]) for k in got] if isinstance(got, dict) else zip(got, want)
    for g, w in pairs:
        np.testing.assert_allclose(g.numpy(), w, rtol=1e-12, atol=1e-12)


@pytest.mark.parametrize("mag", [False, True])
@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("lengths", [None, [9, 0, 4]])
def test_conv(lengths, silu, mag):
    b, L, ch, W = 3, 9, 4, 4
    lengths = None if lengths is None else np.array(lengths)
    args = [rand(b, L, ch, seed=0), rand(ch, W, seed=1), rand(ch, seed=2), rand(b, W - 1, ch, seed=3), lengths, silu]
    both(R.conv, D.conv, args, dict(mag=mag))
    both(R.conv, D.conv, args, dict(mag=mag, dy=rand(b, L, ch, seed=4), dfinal=rand(b, W - 1, ch, seed=5)))


@pytest.mark.parametrize("mag", [False, True])
@pytest.mark.parametrize("soft,gate", [(True, True), (False, False)])
@pytest.mark.parametrize("lengths", [None, [7, 0, 3]])
def test_selective(lengths, soft, gate, mag):
    b, L, ch, G, N = 3, 7, 4, 2, 3
    lengths = None if lengths is None else np.array(lengths)
    dt = rand(b, L, ch, seed=1)
    args = [rand(b, L, ch, seed=0), dt if soft else np.abs(dt), -np.abs(rand(ch, N, seed=2)), rand(b, L, G, N, seed=3),
            rand(b, L, G, N, seed=4), rand(ch, seed=5), rand(b, ch, N, seed=6), lengths]
    kw = dict(soft=soft, bias=rand(ch, seed=7) if soft else None, z=rand(b, L, ch, seed=8) if gate else None, mag=mag)
    both(R.selective, D.selective, args, kw)
    both(R.selective, D.selective, args, dict(kw, dy=rand(b, L, ch, seed=9), dfinal=rand(b, ch, N, seed=10)))
