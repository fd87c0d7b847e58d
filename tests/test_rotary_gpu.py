"""GPU parity of the rotary positions with their 64-bit definition, and the scan that they make turn."""
import pytest
import torch

import block_reference as R
from test_gated_gpu import TYPES, Draw, close, ssd, wide64  # noqa: F401

pytestmark = pytest.mark.gpu

#        type, batch, tokens, heads of each, dim, turned, interleaved, positions, lengths, columns in front, scale
CASES = [("bf16", 2, 33, (1, 1), 128, 128, False, None, None, 0, 1.0),
         ("bf16", 2, 300, (8, 8), 128, 64, True, "start", None, 64, 1.2),
         ("f16", 3, 65, (4, 1), 64, 64, True, "each", [65, 0, 1], 3, 1.0),
         ("f32", 1, 1, (1, 0), 2, 2, False, "start", None, 0, 1.0),
         ("f32", 2, 129, (3, 2), 33, 22, False, "each", [7, 200], 1, 0.5),
         ("f32", 2, 40, (2, 5), 33, 18, True, "start", None, 5, 1.0),
         ("bf16", 1, 5000, (8, 8), 256, 256, False, "start", None, 128, 1.0),   # four heads a thread
         ("f16", 2, 3000, (5, 6), 80, 36, True, None, [3000, 17], 0, 1.1),       # a vector across the turned entries' end
         ("f32", 1, 2000, (32, 8), 128, 128, True, "each", None, 0, 1.0),
         ("bf16", 1, 7, (300, 1), 24, 8, False, None, None, 0, 1.0),
         ("f16", 2, 90, (3, 2), 44, 40, False, "start", None, 4, 1.0),           # vectors of four, of two, none
         ("bf16", 2, 90, (3, 2), 46, 44, True, "start", [90, 3], 2, 1.0),
         ("f32", 2, 90, (3, 2), 46, 44, False, "each", None, 2, 1.0),
         ("f16", 2, 900, (9, 2), 46, 46, False, None, None, 2, 1.0),
         ("bf16", 2, 900, (9, 2), 44, 44, True, None, None, 4, 1.0)]


def make(c, seed=4):
    kind, b, L, heads, dim, turned, interleaved, positions, lengths, before, scale = c
    d, T = Draw(seed), TYPES[kind]
    x = [d.wide((b, L), h * dim, T, before, 0).unflatten(-1, (h, dim)) if h else None for h in heads]
    at = None
    if positions == "start":
        at = torch.tensor([2 ** 31 - 6000, -5, 12][:b], dtype=torch.int32, device="cuda")
    elif positions == "each":
        at = torch.randint(-10, 2 ** 31 - 1, (b, L), generator=d.g, device="cuda", dtype=torch.int64).to(torch.int32)
    f = [10000.0 ** (-2 * k / turned) for k in range(turned // 2)]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if n is not None:
        for t in x:
            for k, m in enumerate(n.tolist()):
                if t is not None:
                    t[k, m:] = float("nan")
    return x, at, n, turned, torch.tensor(f, dtype=torch.float64, device="cuda"), interleaved, scale, T


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("c", CASES)
def test_turned(ssd, c, inverse):  # noqa: F811
    x, at, n, turned, f, interleaved, scale, T = make(c)
    call = ssd.ssd_rotary_backward if inverse else ssd.ssd_rotary_forward
    got = call(*x, ssd.ssd_rotary_table(turned), at, n, interleaved=interleaved, scale=scale)
    got = got if isinstance(got, tuple) else (got,)
    for k, y in enumerate(got):
        assert y.is_contiguous() and y.dtype == T
        t = x[k].double()
        if n is not None:
            t = torch.where(R.kept(*t.shape[:2], n, t)[..., None], t, 0.0)
        close(f"tensor {k}", y, R.rotary(t, f, at, n, interleaved, scale, inverse, fast=T != torch.float32))
        if n is None:
            assert torch.equal(y[..., turned:], x[k][..., turned:]), "the entries past the turned ones are copied"


def test_entries_that_are_copied_may_hold_anything(ssd):  # noqa: F811
    x = torch.ones(1, 3, 2, 32, device="cuda", dtype=torch.bfloat16)
    x[..., 9::2], x[..., 10::2] = float("inf"), float("nan")
    y = ssd.ssd_rotary_forward(x, None, ssd.ssd_rotary_table(6), interleaved=True)
    assert bool(torch.isfinite(y[..., :6]).all()) and torch.equal(y[..., 6:].isnan(), x[..., 6:].isnan())
    assert bool((y[..., 9::2] == float("inf")).all())


def test_back_and_forth_and_shifted(ssd):  # noqa: F811
    """The inverse undoes the turn, and a product of two turned rows depends on their distance alone."""
    d, table = Draw(1), ssd.ssd_rotary_table(64)
    x, y = d.normal(1, 50, 2, 64), d.normal(1, 50, 3, 64)
    at = torch.tensor([10 ** 9], dtype=torch.int32, device="cuda")
    turned = ssd.ssd_rotary_forward(x, y, table, at)
    back = ssd.ssd_rotary_backward(*turned, table, at)
    for a, b in zip(back, (x, y)):  # two turns, each off by at most 17 U of a pair's magnitudes (block_reference)
        assert float((a - b).abs().max()) <= 4 * 17 * R.U * float(b.abs().max()) * 2
    near = ssd.ssd_rotary_forward(x, y, table)
    far, close_by = (torch.einsum("hd,gd->hg", q[0][0, 30], q[1][0, 11]) for q in (turned, near))
    assert float((far - close_by).abs().max()) <= 200 * R.U * float(x[0, 30].norm(dim=-1).max() * y[0, 11].norm(dim=-1).max())


@pytest.mark.parametrize("T", [torch.bfloat16, torch.float32])
def test_tokens_one_by_one(ssd, T):  # noqa: F811
    d, table = Draw(3), ssd.ssd_rotary_table(32)
    B, C = d.normal(3, 9, 2, 40, dtype=T), d.normal(3, 9, 2, 40, dtype=T)
    start = torch.tensor([0, 7, 123456], dtype=torch.int32, device="cuda")
    want = ssd.ssd_rotary_forward(B, C, table, start, interleaved=True, scale=1.5)
    for t in range(9):
        got = ssd.ssd_rotary_step(B[:, t], C[:, t], table, start + t, interleaved=True, scale=1.5)
        assert all(torch.equal(g, w[:, t]) for g, w in zip(got, want))


def test_strides_past_32_bits(ssd):  # noqa: F811
    big = torch.empty(2, 3, 1 << 29, device="cuda", dtype=torch.bfloat16)
    x = big[..., :128].unflatten(-1, (2, 64))
    x.copy_(Draw(1).normal(2, 3, 2, 64, dtype=torch.bfloat16))
    table = ssd.ssd_rotary_table(64)
    assert torch.equal(ssd.ssd_rotary_forward(x, None, table), ssd.ssd_rotary_forward(x.contiguous(), None, table))


def test_streams_and_graphs(ssd):  # noqa: F811
    d, table = Draw(8), ssd.ssd_rotary_table(64)
    B, C = d.normal(2, 70, 1, 64), d.normal(2, 70, 1, 64)
    at = torch.tensor([5, 9], dtype=torch.int32, device="cuda")
    want = ssd.ssd_rotary_forward(B, C, table, at)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    got = ssd.ssd_rotary_forward(B, C, table, at, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.ssd_rotary_step(B[:, 0], C[:, 0], table, at)
    at += 3  # the graph reads the positions when it runs
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ssd.ssd_rotary_step(B[:, 0], C[:, 0], table, at)))


def test_a_layer_whose_state_turns(ssd):  # noqa: F811
    """B and C turned, the scan, and the norm gated by z, against the recurrence with complex decays exp(dt A + i frequency): as a
    prompt, and its last tokens one by one.  bfloat16 throughout, so the tolerance is the scan's own, 1e-2 + 1e-2 |value|, of
    what it takes as B and C (turned and rounded) for the scan; the norm is checked on the scan's rounded output."""
    d, b, L, H, N, P = Draw(12), 2, 320, 4, 64, 64
    T = torch.bfloat16
    x, B, C, z = d.normal(b, L, H, P, dtype=T), d.normal(b, L, 1, N, dtype=T), d.normal(b, L, 1, N, dtype=T), d.normal(b, L, H * P, dtype=T)
    dt, A, w = torch.nn.functional.softplus(d.normal(b, L, H) - 4), -d.normal(H).abs() - 0.5, 1 + d.normal(H * P, scale=0.1)
    table = ssd.ssd_rotary_table(N)
    Bt, Ct = ssd.ssd_rotary_forward(B, C, table)
    y, final = ssd.ssd_forward(x, dt, A, Bt, Ct, None, None, 64)
    out, _, rstd = ssd.ssd_group_norm_forward(y.flatten(2), H, w, z=z, gate_first=True, rms=True)
    # complex states, one for each pair, in the frame that turns with the token
    f = torch.tensor([10000.0 ** (-2 * k / N) for k in range(N // 2)], dtype=torch.float64, device="cuda")
    pair = lambda t: torch.complex(t.double()[..., :N // 2], t.double()[..., N // 2:])[:, :, 0]  # noqa: E731
    state = torch.zeros(b, H, N // 2, P, dtype=torch.complex128, device="cuda")
    ys = []
    for t in range(L):
        decay = torch.exp((dt[:, t].double() * A.double())[..., None] - 1j * f)  # (b, H, N / 2)
        state = decay[..., None] * state + pair(B)[:, t, None, :, None] * (dt[:, t].double()[..., None] * x[:, t].double())[:, :, None]
        ys.append(torch.einsum("bn,bhnp->bhp", pair(C)[:, t].conj(), state).real)
    want = torch.stack(ys, 1)
    # B and C are rounded to bfloat16 once more after the turn: 2^-8 of each product of a B and a C
    mag = torch.zeros(b, H, N, P, dtype=torch.float64, device="cuda")
    size = []
    for t in range(L):
        grow = torch.exp(dt[:, t].double() * A.double())[..., None, None]
        mag = grow * mag + Bt[:, t, 0].double().abs()[:, None, :, None] * (dt[:, t].double()[..., None] * x[:, t].double().abs())[:, :, None]
        size.append(torch.einsum("bn,bhnp->bhp", Ct[:, t, 0].double().abs(), mag))
    tol = 1e-2 + 1e-2 * want.abs() + 2 * 2.0 ** -8 * torch.stack(size, 1)
    assert bool(((y.double() - want).abs() <= tol).all())
    close("norm", out.flatten(0, 1), R.group_norm(y.flatten(2).flatten(0, 1).double(), H, w.double(), None, z.flatten(0, 1).double(), gate_first=True, rms=True)["y"])
    # the last tokens one by one, from the state in front of them
    start = L - 8
    _, state = ssd.ssd_forward(x[:, :start].contiguous(), dt[:, :start].contiguous(), A, Bt[:, :start].contiguous(), Ct[:, :start].contiguous(), None, None, 64)
    for t in range(start, L):
        at = torch.full((b,), t, dtype=torch.int32, device="cuda")
        Bs, Cs = ssd.ssd_rotary_step(B[:, t], C[:, t], table, at)
        assert torch.equal(Bs, Bt[:, t]) and torch.equal(Cs, Ct[:, t])
        y_t = ssd.ssd_step(x[:, t].contiguous(), dt[:, t].contiguous(), A, Bs, Cs, None, state)
        assert bool(((y_t.double() - want[:, t]).abs() <= tol[:, t]).all())
        o_t, _, _ = ssd.ssd_group_norm_forward(y_t.flatten(1), H, w, z=z[:, t], gate_first=True, rms=True)
        assert bool(torch.isfinite(o_t).all())
    # the gradients come back through the norm, the scan and the turn
    do = d.normal(b, L, H * P, dtype=T)
    g = ssd.ssd_group_norm_backward(y.flatten(2), H, w, None, None, rstd, do, z=z, gate_first=True)
    s = ssd.ssd_backward(x, dt, A, Bt, Ct, None, None, g["dx"].unflatten(-1, (H, P)))
    dB, dC = ssd.ssd_rotary_backward(s["dB"], s["dC"], table)
    for got, turned in ((dB, s["dB"]), (dC, s["dC"])):
        close("turned back", got, R.rotary(turned.double(), f, inverse=True))


def test_refusals(ssd):  # noqa: F811
    x, table = torch.zeros(2, 5, 3, 16, device="cuda"), ssd.ssd_rotary_table(16)
    int32 = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_rotary_forward(x, x[..., :8], table)
    with pytest.raises(ValueError, match="dims"):
        ssd.ssd_rotary_forward(x[0], None, table)
    with pytest.raises(TypeError):
        ssd.ssd_rotary_forward(x, x.half(), table)
    with pytest.raises(TypeError):
        ssd.ssd_rotary_forward(x, x, table, int32(2).long())
    with pytest.raises(ValueError, match="positions"):
        ssd.ssd_rotary_forward(x, x, table, int32(2, 4))
    with pytest.raises(ValueError, match="table"):
        ssd.ssd_rotary_forward(x, x, table.cpu())
    with pytest.raises(ssd.SSDError):
        ssd.ssd_rotary_forward(x, x, ssd.ssd_rotary_table(18))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_rotary_forward(x, x, table, scale=float("inf"))
    with pytest.raises(ValueError, match="dense"):
        ssd.ssd_rotary_forward(x.transpose(1, 2), None, table)
