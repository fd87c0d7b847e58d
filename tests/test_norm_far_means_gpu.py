"""The grouped norm's and the layer norm's gradient of rows whose mean is many deviations from zero.

The gradient gets the mean and takes (q - mean) rstd.  That difference is rounded to a float32 of its own size and the product once more,
so xhat is off by at most 2 U of itself (U = 2^-24) however far the mean lies; a form that rounds mean * rstd first is off by up to half
a step of that product instead, the same for the whole group: 512 U at a mean of a thousand deviations."""
import pytest
import torch

import block_reference as R
from test_gated_gpu import Draw, close, ssd  # noqa: F401

pytestmark = pytest.mark.gpu

U = R.U
#        rows, groups, channels of a group, columns in front
SIZES = [(2, 2, 64, 0),      # whole vectors
         (70, 3, 512, 4),    # the same, several threads a group and rows a block
         (2, 3, 30, 1),      # pairs
         (3, 2, 33, 1),      # a half pair at the group's end
         (2, 1, 4096, 0)]    # wider than the registers


def rows_and_stats(rows, groups, per, front, mean):
    d, width = Draw(rows + per), groups * per
    x = d.wide((rows,), width, torch.float32, front, 0)
    x += mean * (1 + 0.1 * torch.arange(groups, device="cuda")).repeat_interleave(per)
    q = x.double().unflatten(-1, (groups, per))
    m = q.mean(-1)
    return d, x, m.float(), torch.rsqrt((q - m[..., None]).square().mean(-1) + 1e-5).float()


def gradients(x, w, dy, mean, rstd):
    """{name: (value, bound)} of a norm's gradients from the statistics as given, g = dy the gradient of xhat w; no gate."""
    rows, groups = mean.shape
    split = lambda t: t.unflatten(-1, (groups, -1))  # noqa: E731
    x, w, dy, mean, rstd = x.double(), w.double(), dy.double(), mean.double()[..., None], rstd.double()[..., None]
    xh = (split(x) - mean) * rstd
    e_xh, gw = 2 * U * xh.abs(), split(dy * w)
    # sums over the group: at most 32 values a thread or one in 256 of a wide group's, then the threads' (as block_reference)
    k = (gw.shape[-1] / 256 + 60) * U
    s1, m1 = gw.mean(-1, keepdim=True), gw.abs().mean(-1, keepdim=True)
    s2, m2 = (gw * xh).mean(-1, keepdim=True), (gw * xh).abs().mean(-1, keepdim=True)
    e_s1, e_s2 = m1 * (k + U), m2 * (k + 3 * U)
    dx = rstd * (gw - s1 - xh * s2)
    e_dx = rstd * (e_s1 + xh.abs() * e_s2 + e_xh * s2.abs() + U * gw.abs() + 6 * U * (gw.abs() + m1 + xh.abs() * m2))
    # a product's rounding and xhat's two; each of the rows is added once
    terms = split(dy).abs() * xh.abs()
    return {"dx": (dx.flatten(1), e_dx.flatten(1)), "dweight": ((split(dy) * xh).sum(0).flatten(), (terms.sum(0) * (rows + 4) * U).flatten())}, xh.flatten(1), e_xh.flatten(1)


@pytest.mark.parametrize("mean", [0.0, 10.0, 1000.0, 10000.0])
@pytest.mark.parametrize("size", SIZES)
def test_groups(ssd, size, mean):  # noqa: F811
    d, x, m, r = rows_and_stats(*size, mean)
    width, groups = x.shape[1], size[1]
    w, b, dy, z = d.normal(width), d.normal(width), d.normal(*x.shape), d.normal(*x.shape)
    want, xh, e_xh = gradients(x, w, dy, m, r)
    got = ssd.ssd_group_norm_backward(x, groups, w, None, m, r, dy)
    for name, value in want.items():
        close(name, got[name], value)
    # behind a gate dz = dy n silu'(z) takes the norm's own value
    got = ssd.ssd_group_norm_backward(x, groups, w, b, m, r, dy, z=z)
    w, b, dy = w.double(), b.double(), dy.double()
    _, _, _, slope, e_slope = R._silu(z.double())
    n, e_n = xh * w + b, e_xh * w.abs() + 2 * U * (xh * w).abs() + U * (xh * w + b).abs()
    close("dz", got["dz"], (dy * n * slope, dy.abs() * (e_n * slope.abs() + n.abs() * (e_slope + 3 * U * slope.abs()))))


@pytest.mark.parametrize("per", [64, 30, 33])
@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16])
def test_16_bits(ssd, T, per):  # noqa: F811
    """Rows of one value only, whose xhat is zero, and the smallest values of the type: dweight = sum dy xhat to its roundings."""
    d, groups = Draw(per), 2
    x = torch.full((3, groups * per), 1000.5, device="cuda").to(T)
    x[1] = torch.randint(-127, 128, (groups * per,), generator=d.g, device="cuda").to(T) * (2.0 ** -24 if T == torch.float16 else 2.0 ** -133)
    x[2] = d.normal(groups * per, dtype=T) + 500
    q = x.double().unflatten(-1, (groups, per))
    m = q.mean(-1).float()
    m[0], m[1] = x[0, 0].float(), 0.0
    r = torch.full_like(m, 316.227766)  # 1 / sqrt(1e-5), where the variance is nothing
    r[1] = 2.0 ** 18 if T == torch.float16 else 2.0 ** 120
    for row in range(3):
        dy, one = d.normal(1, x.shape[1], dtype=T), slice(row, row + 1)
        want, _, _ = gradients(x[one], torch.ones(x.shape[1], device="cuda"), dy, m[one], r[one])
        got = ssd.ssd_group_norm_backward(x[one], groups, torch.ones(x.shape[1], device="cuda"), None, m[one], r[one], dy)
        close("dweight", got["dweight"], want["dweight"])
        if row == 0:
            assert not bool(got["dweight"].any())


@pytest.mark.parametrize("mean", [0.0, 10.0, 1000.0, 10000.0])
@pytest.mark.parametrize("rows, per, front", [(2, 64, 0), (70, 512, 4), (2, 30, 1), (3, 33, 1), (2, 20000, 0)])  # the last wider than the registers
def test_layer_norm(ssd, rows, per, front, mean):  # noqa: F811
    d, x, m, r = rows_and_stats(rows, 1, per, front, mean)
    w, dy = d.normal(per), d.normal(*x.shape)
    want, _, _ = gradients(x, w, dy, m, r)
    got = ssd.ssd_layer_norm_backward(x, w, m[:, 0].contiguous(), r[:, 0].contiguous(), dy)
    for name, value in want.items():
        close(name, got[name], value)


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("per", [64, 33])
def test_layer_norm_of_one_value(ssd, per, T):  # noqa: F811
    """Rows of one value only have an xhat of zero, whatever 1 / sqrt(eps) is."""
    x, dy = torch.full((3, per), 1000.5, device="cuda").to(T), Draw(per).normal(3, per, dtype=T)
    m, r = x[:, 0].float(), torch.full((3,), 316.227766, device="cuda")
    got = ssd.ssd_layer_norm_backward(x, torch.ones(per, device="cuda"), m, r, dy)
    assert not bool(got["dweight"].any())


@pytest.mark.parametrize("per", [64, 30, 33])
@pytest.mark.parametrize("T", [torch.bfloat16, torch.float16, torch.float32])
def test_infinities_and_nans(ssd, T, per):  # noqa: F811
    """With a mean of 0 and an rstd of 1 dweight is dy x: an infinity keeps its sign, a NaN stays one, and the other group is as without."""
    d, groups = Draw(per), 2
    x, dy, one = d.normal(1, groups * per, dtype=T), d.normal(1, groups * per, dtype=T), torch.ones(groups * per, device="cuda")
    m, r = torch.zeros(1, groups, device="cuda"), torch.ones(1, groups, device="cuda")
    clean = ssd.ssd_group_norm_backward(x, groups, one, None, m, r, dy)
    x[0, 4], x[0, 7], x[0, 9] = float("inf"), -float("inf"), float("nan")
    got = ssd.ssd_group_norm_backward(x, groups, one, None, m, r, dy)
    want = dy[0].double() * x[0].double()
    assert got["dweight"][4] == want[4] and got["dweight"][7] == want[7] and bool(got["dweight"][9].isnan())
    finite = torch.isfinite(want)
    assert torch.equal(got["dweight"][finite], clean["dweight"][finite])
    assert torch.equal(got["dx"][:, per:], clean["dx"][:, per:]) and not bool(torch.isfinite(got["dx"][:, :per]).any())
