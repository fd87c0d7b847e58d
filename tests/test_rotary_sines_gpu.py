"""The sines and cosines of float32 tensors' rotary positions, read off the turned pairs (1, 0).

The angle is taken to 2^-32 of a turn, and what is left of it next to a quarter turn is rounded to float32: relative to the sine and to
the cosine there at most U = 2^-24 each, since on [-pi/4, pi/4] both x cos x <= sin x and x sin x <= cos x.  Their evaluation is allowed
two units in the last place, 4 U.  A whole turn rounded to float32 before the quarter is taken out would leave up to 1.6 U of an
absolute error, a large part of a sine near half a turn."""
import math

import pytest
import torch

from test_gated_gpu import ssd  # noqa: F401

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def exact(turns):
    """cos and sin in 64 bits of angles in units of 2^-64 of a turn (int64, modulo 2^64)."""
    quarter = (turns + 2 ** 61) >> 62
    rest = (turns - (quarter << 62)).double() * (2 * math.pi / 2.0 ** 64)
    c, s, quarter = torch.cos(rest), torch.sin(rest), quarter % 4
    pick = lambda *v: torch.stack(v).gather(0, quarter[None])[0]  # noqa: E731
    return pick(c, -s, -c, s), pick(s, c, -s, -c)


def tables():
    g = torch.Generator().manual_seed(1)
    some = torch.randint(-2 ** 63, 2 ** 63 - 1, (512,), generator=g)
    # around the eighths of a turn, at distances from 2^-32 of a turn to 2^-8
    near = torch.stack([torch.randint(-2 ** k, 2 ** k, (16,), generator=g) for k in range(33, 57)]).flatten()
    eighths = torch.arange(-4, 4).repeat_interleave(len(near)) * 2 ** 61
    edges = (torch.arange(-4, 4)[:, None] * 2 ** 61 + torch.tensor([-2 ** 32 - 1, -2 ** 32, -1, 0, 1, 2 ** 32])).flatten()
    return torch.cat([some, near.repeat(8) + eighths, edges])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("position", [1, -1, 3, 2 ** 31 - 1])
def test_sines(ssd, position, interleaved):  # noqa: F811
    table = tables().cuda()
    table = table[:len(table) // 4 * 4]
    n = len(table)
    x = torch.zeros(1, 1, 1, 2 * n, device="cuda")
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    x[..., first] = 1.0
    at = torch.tensor([position], dtype=torch.int32, device="cuda")
    y = ssd.ssd_rotary_forward(x, None, table, at, interleaved=interleaved)[0, 0, 0]
    for name, got, want in zip(("cos", "sin"), (y[first], y[second]), exact(table * position)):
        off = (got.double() - want).abs()
        # the value at an angle that is off by at most t = 2 pi 2^-32 is off by at most t, and its size is at most |want| + t, of which 5 U
        t = 2 * math.pi * 2.0 ** -32
        tol = t + 5 * U * (want.abs() + t)
        assert bool((off <= tol).all()), f"{name}: {int((off > tol).sum())} off, worst {float((off / tol).max()):.3g} of the bound, {float(off.max() / U):.3g} U"
