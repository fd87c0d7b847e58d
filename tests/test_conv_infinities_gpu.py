"""Live infinities through the convolution's gradient, at the tokens that two runs of the kernel share and at a row's length.
Without silu and with terms of one sign the 64-bit definition has one infinity per tap, channel or token, of a certain sign."""
import numpy as np
import pytest
import torch

import layer_reference as R
from test_layer_gpu import TYPES, Draw, np64, spoil, ssd  # noqa: F401
from test_layer_infinities_gpu import agree

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.mark.parametrize("what", ["x", "dy"])
@pytest.mark.parametrize("kind,b,L,ch,W,lengths", [("f32", 1, 40, 6, 4, None), ("bf16", 2, 80, 8, 4, [33, 80]), ("f16", 2, 50, 5, 3, [50, 17]),
                                                   ("f32", 2, 33, 4, 2, [1, 32])])
def test_backward(ssd, kind, b, L, ch, W, lengths, what):  # noqa: F811
    d, T = Draw(23), TYPES[kind]
    some = lambda *shape, dtype=T: (d.normal(*shape).abs() + 0.1).to(dtype)  # noqa: E731
    x, w, bias, init, dy, df = (some(b, L, ch), some(ch, W, dtype=torch.float32), some(ch, dtype=torch.float32), some(b, W - 1, ch),
                                some(b, L, ch), some(b, W - 1, ch))
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    into = x if what == "x" else dy
    # every channel at a token of its own: around the ends of runs of 16 tokens, and the rows' last ones
    ends = [L] * b if lengths is None else lengths
    for c in range(ch):
        for i in range(b):
            into[i, max(0, min(ends[i] - 1 - c % 3, 15 + c // 3)) if c % 2 else ends[i] - 1, c] = INF
    spoil(x, n, NAN)
    spoil(dy, n, NAN)
    out = ssd.ssd_conv_backward(x, w, bias, dy, init, n, silu=False, dfinal=df, want_dinit=True)
    args = [np.nan_to_num(np64(x), nan=0.0, posinf=np.inf), np64(w), np64(bias), np64(init), None if n is None else np64(n), False]
    gy = np.nan_to_num(np64(dy), nan=0.0, posinf=np.inf)
    with np.errstate(invalid="ignore"):
        ref, mag = R.conv(*args, dy=gy, dfinal=np64(df)), R.conv(*args, dy=gy, dfinal=np64(df), mag=True)
    assert what == "dy" or (np.isfinite(ref[0]).all() and np.isinf(ref[1]).any() and np.isfinite(ref[2]).all())
    for i, (name, add) in enumerate((("dx", 0), ("dweight", b * L / 4), ("dbias", b * L / 4), ("dinit", 0))):
        agree(name, out[name], ref[i], mag[i], 2 * W + 12 + add)
