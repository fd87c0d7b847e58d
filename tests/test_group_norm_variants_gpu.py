"""The grouped norm's kernels that test_group_norm_gpu.py's sizes do not reach, with every gate, with and without a mean, and one group
against the layer norm under every gate.

Beside each size: lanes (threads a group), nv (vectors or pairs a thread), the forward kernel (the walk over many rows, or the one with
that many held), groups a block has room for side by side (more than there are: idle ones) and rows at once; the gradient has
the same lanes, nv and places where it is not said otherwise."""
import pytest
import torch

import block_reference as R
import test_group_norm_gpu as base
from test_gated_gpu import Draw, close, ssd, wide64  # noqa: F401

pytestmark = pytest.mark.gpu

#        type, rows, groups, channels of a group, columns around, weight, bias
SIZES = [("bf16", 2100, 8, 512, (64, 8), True, False),    # 32, 2: walk, 8 groups by 1 row
         ("bf16", 32001, 1, 64, (0, 0), True, True),      # 8, 1: walk, 1 by 32 rows, the last ones past the end
         ("bf16", 40001, 3, 16, (0, 0), True, True),      # 2, 1: walk, 4 (one idle) by 32 rows
         ("bf16", 20003, 3, 128, (8, 0), True, False),    # 8, 2: walk, 4 (one idle) by 8 rows
         ("bf16", 1300, 3, 512, (0, 0), True, True),      # 64, 1: walk, 4 (one idle) by 1 row, several warps a group
         ("f32", 6007, 5, 48, (4, 4), True, True),        # 8, 2 with idle lanes: walk, 8 (three idle) by 4 rows
         ("f32", 1700, 1, 2048, (0, 0), False, True),     # 256, 2: walk, a block a row
         ("f16", 9001, 1, 264, (0, 0), True, True),       # 32, 2 with idle lanes: walk, 1 by 8 rows
         ("f16", 3554, 15, 102, (0, 3), True, True),      # 8, 7: pairs, eight held; 16 (one idle) by 2 rows
         ("f16", 3554, 15, 101, (0, 3), True, True),      # the same with half a pair at a group's end
         ("f32", 12001, 6, 60, (0, 1), True, False),      # 4, 8: pairs, eight held; 8 (two idle) by 8 rows
         ("bf16", 5, 2, 4000, (0, 1), True, True),        # 256, 8: pairs, eight held, a block a group
         ("bf16", 5, 1, 6144, (0, 0), True, True),        # 256, 3: four vectors held; gradient of wide groups
         ("f32", 5, 1, 4096, (4, 0), True, True)]         # 256, 4: four vectors held; gradient of wide groups


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gate", base.GATES)
@pytest.mark.parametrize("c", SIZES)
def test_forward_and_backward(ssd, c, gate, rms):  # noqa: F811
    base.test_forward_and_backward(ssd, c, gate, rms)


@pytest.mark.parametrize("gate", base.GATES)
@pytest.mark.parametrize("width", [256, 250, 33])
def test_one_group_is_the_layer_norm_under_its_gate(ssd, width, gate):  # noqa: F811
    """The layer norm's output (of x silu(z) where the gate comes first) through the activation, against the grouped norm's bounds."""
    d = Draw(width)
    x, z, w, b = d.normal(3, 5, width), d.normal(3, 5, width), d.normal(width), d.normal(width)
    gated, first = gate in ("after", "before"), gate == "before"
    y, mean, rstd = ssd.ssd_group_norm_forward(x, 1, w, b, z=z if gated else None, gate_first=first, silu=gate == "silu")
    assert y.shape == x.shape and mean.shape == rstd.shape == (3, 5, 1)
    silu = lambda t: t * torch.sigmoid(t)  # noqa: E731
    q = (x.double() * silu(z.double())).float() if first else x
    n, wmean, wrstd = ssd.ssd_layer_norm_forward(q, w, b)
    want = silu(n.double()) if gate == "silu" else n.double() * silu(z.double()) if gate == "after" else n.double()
    x64, w64, b64, z64 = wide64(x.flatten(0, 1), w, b, z.flatten(0, 1) if gated else None)
    bound = R.group_norm(x64, 1, w64, b64, z64, gate_first=first, silu=gate == "silu")
    # each of the two norms is within its bound of the definition; the layer norm's rounding of q and n is within the same
    for name, got, other in (("y", y, want), ("mean", mean, wmean[..., None].double()), ("rstd", rstd, wrstd[..., None].double())):
        close(name, got.flatten(0, 1), (other.flatten(0, 1), 2 * bound[name][1]))
