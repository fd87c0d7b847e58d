"""GPU parity of the grouped norm and its gradient with their 64-bit definitions (bounds in block_reference.py)."""
import pytest
import torch

import block_reference as R
from test_gated_gpu import TYPES, Draw, close, ssd, wide64  # noqa: F401

pytestmark = pytest.mark.gpu

#        type, rows, groups, channels of a group, columns around, weight, bias
SIZES = [("f32", 1, 1, 1, (0, 0), True, True),
         ("bf16", 3, 1, 64, (0, 0), True, True),
         ("bf16", 70, 8, 512, (64, 8), True, False),        # a warp a group
         ("f16", 33, 15, 102, (0, 3), True, True),          # odd columns
         ("f32", 9, 3, 24, (4, 4), False, True),
         ("f32", 257, 64, 8, (0, 0), True, True),           # narrow groups, many a block
         ("bf16", 5, 2, 4096, (8, 0), True, True),
         ("f16", 4, 1, 16384, (0, 0), True, True),          # wider than the registers
         ("f32", 3, 2, 4999, (1, 0), True, False),          # the same, odd
         ("bf16", 6000, 4, 64, (0, 0), True, True),
         ("f32", 2, 1, 9001, (0, 0), True, True),           # odd and wider than the registers
         ("bf16", 4000, 2, 40, (8, 8), True, True),
         ("f32", 3000, 1, 130, (0, 0), True, False),
         ("f32", 1500, 2, 1024, (0, 0), True, True),        # several warps a group, many rows a block
         ("bf16", 2500, 1, 2048, (0, 8), True, False),
         ("bf16", 1, 1, 4096, (0, 0), False, False),
         ("f16", 2, 7, 1, (2, 1), True, True)]
GATES = ["none", "silu", "after", "before"]


def make(c, gate, seed=3):
    kind, rows, groups, per, (before, after), weight, bias = c
    d, T, width = Draw(seed), TYPES[kind], groups * per
    x, z = d.wide((rows,), width, T, before, after), d.wide((rows,), width, T, after, before)
    x += (0.5 * torch.linspace(-1, 1, width, device="cuda")).to(T)
    return x, groups, d.normal(width) if weight else None, d.normal(width) if bias else None, z if gate in ("after", "before") else None, d, T


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("c", SIZES)
def test_forward_and_backward(ssd, c, gate, rms):  # noqa: F811
    x, groups, w, b, z, d, T = make(c, gate)
    how = dict(gate_first=gate == "before", silu=gate == "silu")
    y, mean, rstd = ssd.ssd_group_norm_forward(x, groups, w, b, z=z, rms=rms, eps=1e-5, **how)
    x64, w64, b64, z64 = wide64(x, w, b, z)
    want = R.group_norm(x64, groups, w64, b64, z64, rms=rms, **how)
    assert y.dtype == T and rstd.dtype == torch.float32 and (mean is None) == rms
    close("y", y, want["y"])
    close("rstd", rstd, want["rstd"])
    if not rms:
        close("mean", mean, want["mean"])
    wide = d.normal(*x.shape[:1], x.shape[1] + 8, dtype=T)
    dy = wide[:, 8:]
    got = ssd.ssd_group_norm_backward(x, groups, w, b, mean, rstd, dy, z=z, **how)
    want = R.group_norm(x64, groups, w64, b64, z64, rms=rms, stats=wide64(mean, rstd), dy=dy.double(), **how)
    close("dx", got["dx"], want["dx"])
    for k, there in (("dz", z is not None), ("dweight", w is not None), ("dbias", b is not None)):
        if there:
            close(k, got[k], want[k])
        else:
            assert got.get(k) is None
    again = ssd.ssd_group_norm_backward(x, groups, w, b, mean, rstd, dy, z=z, **how)
    assert all(torch.equal(again[k], got[k]) for k in got if got[k] is not None)


@pytest.mark.parametrize("gate", GATES)
def test_one_group_is_the_layer_norm(ssd, gate):  # noqa: F811
    """With one group and no gate the values are those of ssd_layer_norm_forward; and rows may be of any leading shape."""
    d = Draw(7)
    x, w, b = d.normal(3, 5, 256), d.normal(256), d.normal(256)
    y, mean, rstd = ssd.ssd_group_norm_forward(x, 1, w, b, silu=gate == "silu")
    assert mean.shape == rstd.shape == (3, 5, 1) and y.shape == x.shape
    want, wmean, wrstd = ssd.ssd_layer_norm_forward(x, w, b)
    if gate == "none":
        assert torch.equal(y, want) and torch.equal(mean[..., 0], wmean) and torch.equal(rstd[..., 0], wrstd)


@pytest.mark.parametrize("gate", GATES)
@pytest.mark.parametrize("rms", [False, True])
def test_gradient_is_the_slope(ssd, gate, rms):  # noqa: F811
    """Against central differences of the 64-bit definition along a random direction of each input."""
    d, rows, groups, width = Draw(5), 6, 4, 96
    t = {"x": d.normal(rows, width), "weight": d.normal(width), "bias": d.normal(width), "z": d.normal(rows, width)}
    gated, how = gate in ("after", "before"), dict(gate_first=gate == "before", silu=gate == "silu")
    if not gated:
        t.pop("z")
    dy = d.normal(rows, width)
    _, mean, rstd = ssd.ssd_group_norm_forward(t["x"], groups, t["weight"], t["bias"], z=t.get("z"), rms=rms, **how)
    got = ssd.ssd_group_norm_backward(t["x"], groups, t["weight"], t["bias"], mean, rstd, dy, z=t.get("z"), **how)

    def loss(v):
        return float((R.group_norm(v["x"], groups, v["weight"], v["bias"], v.get("z"), rms=rms, **how)["y"][0] * dy.double()).sum())
    for name in t:
        way, step = d.normal(*t[name].shape).double(), 1e-5
        ahead, back = ({k: v.double() + (s * step * way if k == name else 0) for k, v in t.items()} for s in (1, -1))
        slope, terms = (loss(ahead) - loss(back)) / (2 * step), got["d" + name].double() * way
        # float32 sums of 24 to 96 terms stay within 1e-5 of their terms; the differences truncate at about step^2
        assert abs(float(terms.sum()) - slope) <= 1e-5 * float(terms.abs().sum()) + 1e-6 * abs(slope), name


def test_rows_next_to_a_bad_one(ssd):  # noqa: F811
    """An infinity or a NaN stays in its own group."""
    d = Draw(2)
    x, z, w = d.normal(40, 128), d.normal(40, 128), d.normal(128)
    x[3, 5], x[7, 70], z[9, 127] = float("inf"), float("nan"), float("nan")
    y, mean, rstd = ssd.ssd_group_norm_forward(x, 4, w, z=z, gate_first=True)
    bad = torch.zeros(40, 4, dtype=torch.bool, device="cuda")
    bad[3, 0] = bad[7, 2] = bad[9, 3] = True
    finite = torch.isfinite(y).unflatten(1, (4, 32))
    assert bool(finite.all(-1)[~bad].all()) and not bool(finite.all(-1)[bad].any())
    got = ssd.ssd_group_norm_backward(x, 4, w, None, mean, rstd, d.normal(40, 128), z=z, gate_first=True)
    assert bool(torch.isfinite(got["dx"]).unflatten(1, (4, 32)).all(-1)[~bad].all())
    assert bool(torch.isfinite(got["dweight"][32:64]).all())


def test_long_rows_of_strides(ssd):  # noqa: F811
    """A row stride that passes 2^31 elements within the tensor."""
    big = torch.empty(3, 1 << 30, device="cuda", dtype=torch.bfloat16)
    x = big[:, :256]
    x.copy_(Draw(1).normal(3, 256, dtype=torch.bfloat16))
    y, _, _ = ssd.ssd_group_norm_forward(x, 2)
    assert torch.equal(y, ssd.ssd_group_norm_forward(x.contiguous(), 2)[0])


def test_streams_and_graphs(ssd):  # noqa: F811
    d = Draw(6)
    x, z, w, b, dy = d.normal(300, 256), d.normal(300, 256), d.normal(256), d.normal(256), d.normal(300, 256)
    y, mean, rstd = ssd.ssd_group_norm_forward(x, 8, w, b, z=z)
    want = ssd.ssd_group_norm_backward(x, 8, w, b, mean, rstd, dy, z=z)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2, mean2, rstd2 = ssd.ssd_group_norm_forward(x, 8, w, b, z=z, stream=other)
    got = ssd.ssd_group_norm_backward(x, 8, w, b, mean2, rstd2, dy, z=z, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(y, y2) and all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.ssd_group_norm_backward(x, 8, w, b, mean, rstd, dy, z=z)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)


@pytest.mark.parametrize("width", [64, 30])
def test_the_c_entry_gives_dbias_without_a_bias(ssd, width):  # noqa: F811
    """dbias is the sum of n's gradient whether or not a bias was added."""
    from state_space_sequence_ssd_gb300 import _ffi
    d, rows = Draw(14), 50
    x, w, dy = d.normal(rows, width), d.normal(width), d.normal(rows, width)
    _, mean, rstd = ssd.ssd_group_norm_forward(x, 2, w)
    want = ssd.ssd_group_norm_backward(x, 2, w, torch.zeros(width, device="cuda"), mean, rstd, dy)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.full_like(w, float("nan"))
    p = lambda t: t.data_ptr()  # noqa: E731
    assert _ffi.lib().ssd_group_norm_backward(_ffi.SSD_F32, p(x), width, None, 0, p(w), None, 0, p(mean), p(rstd), p(dy), width, rows, width, 2, p(dx), None,
                                              p(dw), p(db), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(dx, want["dx"]) and torch.equal(dw, want["dweight"]) and torch.equal(db, want["dbias"])
    db.fill_(float("nan"))  # and alone
    assert _ffi.lib().ssd_group_norm_backward(_ffi.SSD_F32, p(x), width, None, 0, p(w), None, 0, p(mean), p(rstd), p(dy), width, rows, width, 2, p(dx), None,
                                              None, p(db), torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(db, want["dbias"])


@pytest.mark.parametrize("rms", [False, True])
def test_groups_of_several_warps_over_many_rows(ssd, rms):  # noqa: F811
    """Rows that follow one another in a block do not meet in the sums: rows of sizes far apart, many times."""
    d = Draw(15)
    x = d.normal(6000, 4096, dtype=torch.bfloat16) * torch.exp2((torch.arange(6000, device="cuda") % 13 - 6.0))[:, None].to(torch.bfloat16)
    q = x.double()
    mean = q.mean(-1, keepdim=True) * (not rms)
    want = 1 / torch.sqrt((q - mean).square().mean(-1, keepdim=True) + 1e-5)
    first = ssd.ssd_group_norm_forward(x, 1, rms=rms)
    # as block_reference: 16 + 60 additions of 2^-24 and the root's
    assert float(((first[2].double() - want).abs() / want).max()) <= 90 * R.U
    for _ in range(20):
        again = ssd.ssd_group_norm_forward(x, 1, rms=rms)
        assert torch.equal(again[0], first[0]) and torch.equal(again[2], first[2])


def test_one_row_as_a_vector(ssd):  # noqa: F811
    d = Draw(16)
    x, z, w, dy = d.normal(96), d.normal(96), d.normal(96), d.normal(96)
    y, mean, rstd = ssd.ssd_group_norm_forward(x, 3, w, z=z)
    want = ssd.ssd_group_norm_forward(x[None], 3, w, z=z[None])
    assert y.shape == (96,) and mean.shape == rstd.shape == (3,) and all(torch.equal(a, b[0]) for a, b in zip((y, mean, rstd), want))
    g = ssd.ssd_group_norm_backward(x, 3, w, None, mean, rstd, dy, z=z)
    assert g["dx"].shape == g["dz"].shape == (96,) and g["dweight"].shape == (96,) and g["dbias"] is None


def test_refusals(ssd):  # noqa: F811
    x = torch.zeros(4, 96, device="cuda")
    with pytest.raises(ValueError, match="divide"):
        ssd.ssd_group_norm_forward(x, 5)
    with pytest.raises(ValueError, match="exclude"):
        ssd.ssd_group_norm_forward(x, 3, z=x, silu=True)
    with pytest.raises(ValueError, match="gate"):
        ssd.ssd_group_norm_forward(x, 3, gate_first=True)
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_group_norm_forward(x, 3, z=x[:, :48])
    with pytest.raises(TypeError):
        ssd.ssd_group_norm_forward(x, 3, z=x.half())
    with pytest.raises(ValueError, match="evenly"):
        ssd.ssd_group_norm_forward(torch.zeros(3, 4, 96, device="cuda")[:, :2], 3)
    with pytest.raises(ssd.SSDError):
        ssd.ssd_group_norm_forward(x, 3, eps=-1.0)
