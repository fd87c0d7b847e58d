"""Norms of rows that hold one value only: the sum of such a row is exact here (the value has 10 bits, the row at most 2^13 channels), so
its mean is the value itself and the output the bias.  A mean that is a rounding further off than the sum's would be scaled by
1 / sqrt(eps) = 316 and shift the whole group."""
import pytest
import torch

from test_gated_gpu import TYPES, Draw, ssd  # noqa: F401

pytestmark = pytest.mark.gpu

VALUE = {"bf16": 996.0, "f16": 1000.5, "f32": 1000.5}
#        rows, groups, channels of a group, columns in front
SIZES = [(3, 2, 96, 0), (5, 1, 33, 1), (4, 3, 102, 3), (3000, 1, 2040, 0), (20003, 3, 56, 8), (3, 1, 5000, 0), (3, 2, 3999, 1), (2, 1, 8001, 0), (3, 1, 7000, 0)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("kind", list(TYPES))
def test_groups(ssd, kind, size):  # noqa: F811
    rows, groups, per, front = size
    d, T, width = Draw(per), TYPES[kind], groups * per
    x = d.wide((rows,), width, T, front, 0)
    x.copy_(VALUE[kind] * torch.exp2(torch.arange(groups, device="cuda").float()).repeat_interleave(per).expand(rows, -1))
    w, b = d.normal(width), d.normal(width)
    y, mean, rstd = ssd.ssd_group_norm_forward(x, groups, w, b)
    assert torch.equal(mean, x[:, ::per].float())
    assert torch.equal(y, b.to(T).expand(rows, -1))
    # two roundings and the reciprocal root's
    assert float((rstd.double() / 1e-5 ** -0.5 - 1).abs().max()) <= 8 * 2.0 ** -24


@pytest.mark.parametrize("size", [(4, 2, 96, 0), (4, 2, 33, 1), (4, 1, 9001, 1)])
def test_infinite_sums(ssd, size):  # noqa: F811
    """A group with an infinity has that as its mean, one with both or a NaN has a NaN; a sum next to the largest float32 is still one."""
    rows, groups, per, front = size
    x = Draw(1).wide((rows,), groups * per, torch.float32, front, 0)
    x[0, 3], x[1, 3] = float("inf"), -float("inf")
    x[2, 3], x[2, 5] = float("inf"), -float("inf")
    x[3] = 0.0
    x[3, 7] = 3.4e38
    mean = ssd.ssd_group_norm_forward(x, groups)[1]
    assert mean[0, 0] == float("inf") and mean[1, 0] == -float("inf") and bool(mean[2, 0].isnan())
    assert abs(float(mean[3, 0]) / (float(x[3, 7]) / per) - 1) <= 2.0 ** -23
