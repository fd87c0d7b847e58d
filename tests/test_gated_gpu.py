"""GPU parity of the gated linear recurrence with its 64-bit definition (block_reference.py has the bounds of a float32
evaluation; a result is then rounded once to its type, by at most half its epsilon)."""
import pytest
import torch

import block_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ssd():
    from state_space_sequence_ssd_gb300 import build
    build.build()
    import state_space_sequence_ssd_gb300 as m
    m.ssd_get_device_error()
    yield m
    assert m.ssd_get_device_error() == 0


def close(name, got, want):
    value, bound = want
    assert got.shape == value.shape, (name, got.shape, value.shape)
    assert torch.isfinite(got).all(), name
    # half a step of the type, and half a step of float16's subnormals
    tol = bound + (value.abs() + bound) * torch.finfo(got.dtype).eps / 2 + (2.0 ** -25 if got.dtype == torch.float16 else 2.0 ** -126)
    off = (got.double() - value).abs()
    assert bool((off <= tol).all()), f"{name}: {int((off > tol).sum())} of {off.numel()} off, worst {float((off / tol).max()):.3g} of the bound"


class Draw:
    def __init__(self, seed):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)

    def normal(self, *shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype)

    def wide(self, rows, n, T, before, after, scale=1.0):
        """(*rows, n) as a column slice of wider rows; the columns around it are NaN."""
        t = torch.full((*rows, before + n + after), float("nan"), device="cuda", dtype=T)
        t[..., before:before + n] = self.normal(*rows, n, dtype=T, scale=scale)
        return t[..., before:before + n]


def wide64(*t):
    return [None if v is None else v.double() if v.is_floating_point() else v for v in t]


#        type, batch, tokens, channels, init, lengths, columns around the gates, size of the gates, decays
CASES = [("f32", 1, 1, 1, True, None, (0, 0), 1.0, (0.01, 1.0)),
         ("bf16", 2, 7, 8, True, None, (0, 0), 1.0, (0.01, 1.0)),
         ("bf16", 3, 64, 64, False, None, (64, 8), 1.0, (0.01, 1.0)),
         ("f16", 3, 65, 37, True, [65, 0, 64], (3, 2), 2.0, (0.001, 3.0)),
         ("f32", 5, 130, 66, True, [1, 130, 129, 0, 63], (1, 0), 1.0, (1e-6, 30.0)),
         ("f32", 1, 512, 256, True, None, (0, 0), 1.0, (0.008, 0.84)),
         ("bf16", 2, 1000, 200, True, [999, 1000], (8, 8), 1.0, (0.008, 0.84)),
         ("f16", 2, 3001, 16, False, None, (0, 0), 1.0, (0.0001, 0.1)),
         ("f32", 2, 140, 10, True, None, (0, 0), 3.0, (60.0, 300.0)),       # decays below the smallest float32
         # (warps a block and blocks a cluster of the forward pass; of the gradient)
         ("f32", 40, 300, 130, True, None, (2, 0), 30.0, (0.01, 10.0)),     # 4 and 5; 4 and 3
         ("bf16", 75, 200, 128, False, None, (0, 0), 1.0, (0.01, 1.0)),     # 4 and 4; 4 and 2
         ("bf16", 300, 70, 72, True, None, (0, 0), 1.0, (0.01, 1.0)),       # 8 and 1; 4 and 1
         ("f16", 260, 129, 65, True, None, (1, 1), 1.0, (0.01, 1.0)),       # 8 and 1; 4 and 1
         ("bf16", 50, 1300, 64, True, None, (8, 0), 1.0, (0.01, 1.0)),      # 8 and 6; 4 and 6
         ("f32", 24, 1100, 64, True, [(97 * k) % 1101 for k in range(24)], (4, 0), 1.0, (0.01, 1.0)),  # 8 and 8; 4 and 8
         ("f16", 1, 5000, 40, False, [4242], (0, 0), 1.0, (0.001, 0.1)),    # 8 and 8; 8 and 8
         ("f32", 2, 2500, 70, True, [2500, 1030], (1, 0), 1.0, (0.001, 0.1))]  # 8 and 8; 8 and 8


def make(c, seed=5):
    kind, b, L, ch, init, lengths, (before, after), size, (lo, hi) = c
    d, T = Draw(seed), TYPES[kind]
    x, r, i = d.wide((b, L), ch, T, after, before), d.wide((b, L), ch, T, before, after, size), d.wide((b, L), ch, T, before, after, size)
    if lengths is None and b > 100:
        lengths = [(7 * k) % (L + 1) for k in range(b)]
    n = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    if n is not None:
        for t in (x, r, i):
            for k, m in enumerate(n.tolist()):
                t[k, m:] = float("nan")
    A = -torch.exp(torch.linspace(torch.tensor(lo).log(), torch.tensor(hi).log(), ch, device="cuda"))
    return x, r, i, A, d.normal(b, ch) if init else None, n, d, T


@pytest.mark.parametrize("c", CASES)
def test_forward(ssd, c):
    x, r, i, A, init, n, _, T = make(c)
    y, final, states = ssd.ssd_gated_forward(x, r, i, A, init, n, want_states=True)
    want = R.gated(*wide64(x, r, i, A, init), n)
    assert y.dtype == T and final.dtype == states.dtype == torch.float32
    close("y", y, want["y"])
    close("final", final, want["final"])
    close("states", states, want["states"])
    again, none, nothing = ssd.ssd_gated_forward(x, r, i, A, init, n, want_final=False)
    assert none is None and nothing is None and torch.equal(again, y)


@pytest.mark.parametrize("c", CASES)
@pytest.mark.parametrize("given", [False, True])
def test_backward(ssd, c, given):
    x, r, i, A, init, n, d, T = make(c)
    b, L, ch = x.shape
    dy, dfinal = d.normal(b, L, ch, dtype=T), d.normal(b, ch) if init is not None else None
    if n is not None:
        for k, m in enumerate(n.tolist()):
            dy[k, m:] = float("inf")
    states = ssd.ssd_gated_forward(x, r, i, A, init, n, want_states=True)[2] if given else None
    got = ssd.ssd_gated_backward(x, r, i, A, dy, None if given else init, n, states=states, dfinal=dfinal, want_dinit=True)
    want = R.gated(*wide64(x, r, i, A, init), n, dy=dy.double(), dfinal=None if dfinal is None else dfinal.double())
    for k in ("dx", "dr", "di", "dA", "dinit"):
        close(k, got[k], want[k])
    assert got["dx"].dtype == got["dr"].dtype == got["di"].dtype == T
    again = ssd.ssd_gated_backward(x, r, i, A, dy, init, n, dfinal=dfinal)
    assert again["dinit"] is None and all(torch.equal(again[k], got[k]) for k in ("dx", "dr", "di", "dA"))


@pytest.mark.parametrize("c", [("bf16", 5, 4096, (0, 0), False), ("f16", 7, 37, (3, 0), True), ("f32", 300, 130, (2, 1), True), ("bf16", 1, 1, (0, 0), True)])
def test_step(ssd, c):
    kind, b, ch, (before, after), slots = c
    d, T = Draw(11), TYPES[kind]
    x, r, i = (d.wide((b,), ch, T, before, after) for _ in range(3))
    A, pool = -d.normal(ch).abs() - 0.001, d.normal(b + 3, ch)
    at = torch.randperm(b + 3, generator=d.g, device="cuda")[:b].to(torch.int32) if slots else None
    if slots and b > 2:
        at[1] = -1
    state = pool.clone()
    y = ssd.ssd_gated_step(x, r, i, A, state, at)
    rows = torch.arange(b, device="cuda") if at is None else at.long()
    live = rows >= 0
    want = R.gated(*wide64(x[:, None], r[:, None], i[:, None], A, pool[rows.clamp(min=0)]))
    value, bound = (torch.where(live[:, None], q[:, 0], 0.0) for q in want["y"])
    close("y", y, (value, bound))
    close("state", state[rows[live]], (value[live], bound[live]))
    rest = torch.ones(b + 3, dtype=torch.bool, device="cuda")
    rest[rows[live]] = False
    assert torch.equal(state[rest], pool[rest])


def test_prompt_then_tokens_is_one_row(ssd):
    d, b, L, ch = Draw(2), 2, 200, 72
    x, r, i, A = d.normal(b, L, ch), d.normal(b, L, ch), d.normal(b, L, ch), -d.normal(ch).abs()
    y, final, _ = ssd.ssd_gated_forward(x, r, i, A)
    start, state, _ = ssd.ssd_gated_forward(x[:, :190], r[:, :190], i[:, :190], A)
    steps = [ssd.ssd_gated_step(x[:, t], r[:, t], i[:, t], A, state) for t in range(190, L)]
    want = R.gated(*wide64(x, r, i, A))
    close("y", torch.cat([start, torch.stack(steps, 1)], 1), want["y"])
    close("final", state, want["final"])


def test_gradient_is_the_slope(ssd):
    """Central differences of the 64-bit definition along a random direction of every input."""
    d, b, L, ch = Draw(4), 2, 150, 16
    t = {"x": d.normal(b, L, ch), "r": d.normal(b, L, ch), "i": d.normal(b, L, ch), "A": -d.normal(ch).abs() - 0.05, "init": d.normal(b, ch)}
    dy, dfinal = d.normal(b, L, ch), d.normal(b, ch)
    got = ssd.ssd_gated_backward(t["x"], t["r"], t["i"], t["A"], dy, t["init"], dfinal=dfinal, want_dinit=True)

    def loss(v):
        out = R.gated(v["x"], v["r"], v["i"], v["A"], v["init"])
        return float((out["y"][0] * dy.double()).sum() + (out["final"][0] * dfinal.double()).sum())
    for name in t:
        way = d.normal(*t[name].shape).double()
        step = 1e-5
        ahead, back = ({k: v.double() + (s * step * way if k == name else 0) for k, v in t.items()} for s in (1, -1))
        slope = (loss(ahead) - loss(back)) / (2 * step)
        terms = got["d" + name].double() * way
        # the gradient's own bound is far below this: 1e-5 of its terms, and the differences' truncation
        assert abs(float(terms.sum()) - slope) <= 1e-5 * float(terms.abs().sum()) + 1e-6 * abs(slope), name


@pytest.mark.parametrize("T", [torch.float32, torch.bfloat16])
def test_shut_and_open_gates(ssd, T):
    """Gates whose exponentials overflow, or leave nothing, and infinities among them."""
    d, b, L, ch = Draw(8), 1, 140, 16
    x, r, i, A = d.normal(b, L, ch, dtype=T), d.normal(b, L, ch, dtype=T), d.normal(b, L, ch, dtype=T), -d.normal(ch).abs() - 0.01
    for k, v in enumerate([50.0, -50.0, 85.0, -85.0, 200.0, -200.0, float("inf"), float("-inf")]):
        r[0, 10 + 16 * k, :8] = v
        i[0, 18 + 16 * k, 4:12] = v
    y, final, _ = ssd.ssd_gated_forward(x, r, i, A)
    lim = lambda t: t.double().clamp(-1000, 1000)  # noqa: E731  (the definition's bounds count the argument)
    want = R.gated(x.double(), lim(r), lim(i), A.double())
    close("y", y, want["y"])
    dy = d.normal(b, L, ch, dtype=T)
    got = ssd.ssd_gated_backward(x, r, i, A, dy)
    want = R.gated(x.double(), lim(r), lim(i), A.double(), dy=dy.double())
    for k in ("dx", "dr", "di", "dA"):
        close(k, got[k], want[k])


def test_infinities_and_nans_reach_what_the_recurrence_carries_them_to(ssd):
    d, b, L, ch = Draw(9), 1, 700, 8
    x, r, i, A = d.normal(b, L, ch), d.normal(b, L, ch), d.normal(b, L, ch), -torch.full((ch,), 3.0, device="cuda")
    x[0, 100, 1] = float("inf")
    x[0, 300, 2] = float("nan")
    i[0, 301, 3] = float("nan")
    y, final, _ = ssd.ssd_gated_forward(x, r, i, A)
    assert bool((y[0, 100:, 1] == float("inf")).all()) and bool(torch.isfinite(y[0, :100, 1]).all())
    assert bool(y[0, 300:, 2].isnan().all()) and bool(torch.isfinite(y[0, :300, 2]).all())
    assert bool(y[0, 301:, 3].isnan().all()) and bool(torch.isfinite(y[0, :301, 3]).all())
    assert bool(torch.isfinite(y[..., [0, 4, 5, 6, 7]]).all()) and float(final[0, 1]) == float("inf")
    dy = d.normal(b, L, ch)
    dy[0, 400, 5] = float("inf")
    got = ssd.ssd_gated_backward(x, r, i, A, dy)
    assert bool(got["dx"][0, :401, 5].isinf().all()) and bool(torch.isfinite(got["dx"][0, 401:, 5]).all())
    assert bool(torch.isfinite(got["dx"][0, :, 3][:301]).all()), "a NaN of one gate does not reach the gradients of earlier tokens"
    assert bool(torch.isfinite(got["dA"][[0, 4, 6, 7]]).all())


def test_streams_and_graphs(ssd):
    d, b, L, ch = Draw(3), 2, 300, 64
    x, r, i, A, dy = d.normal(b, L, ch), d.normal(b, L, ch), d.normal(b, L, ch), -d.normal(ch).abs() - 0.1, d.normal(b, L, ch)
    y, final, states = ssd.ssd_gated_forward(x, r, i, A, want_states=True)
    grads = ssd.ssd_gated_backward(x, r, i, A, dy)
    state = torch.zeros(b, ch, device="cuda")
    token = ssd.ssd_gated_step(x[:, 0], r[:, 0], i[:, 0], A, state)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    y2, final2, states2 = ssd.ssd_gated_forward(x, r, i, A, want_states=True, stream=other)
    grads2 = ssd.ssd_gated_backward(x, r, i, A, dy, states=states2, stream=other)
    state2 = torch.zeros(b, ch, device="cuda")
    other.wait_stream(torch.cuda.current_stream())
    token2 = ssd.ssd_gated_step(x[:, 0], r[:, 0], i[:, 0], A, state2, stream=other)
    torch.cuda.current_stream().wait_stream(other)
    assert torch.equal(y, y2) and torch.equal(final, final2) and torch.equal(states, states2)
    assert torch.equal(token, token2) and torch.equal(state, state2)
    assert all(torch.equal(grads[k], grads2[k]) for k in ("dx", "dr", "di", "dA"))
    graphs = []
    for _ in range(2):  # two graphs whose workspaces are their own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = ssd.ssd_gated_backward(x, r, i, A, dy)
        graphs.append((g, out))
    for g, out in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for _, out in graphs:
        assert all(torch.equal(grads[k], out[k]) for k in ("dx", "dr", "di", "dA"))


def test_a_slot_past_the_pool_is_reported(ssd):
    x, A = torch.ones(2, 8, device="cuda"), -torch.ones(8, device="cuda")
    state = torch.zeros(3, 8, device="cuda")
    y = ssd.ssd_gated_step(x, x, x, A, state, torch.tensor([3, 1], dtype=torch.int32, device="cuda"))
    assert ssd.ssd_get_device_error() == 8 and ssd.ssd_get_device_error() == 0
    assert bool((y[0] == 0).all()) and bool((y[1] != 0).all()) and bool((state[[0, 2]] == 0).all())


def test_a_wait_that_runs_out_is_reported(ssd):
    """A cluster's exchange that never completes: the kernel gives up, says so, and the next call is right."""
    from state_space_sequence_ssd_gb300 import _ffi
    lib = _ffi.lib()
    kinds = {lib.ssd_kernel_name(k).decode(): k for k in range(32)}
    d, b, L, ch = Draw(13), 2, 1000, 64
    x, r, i, A, dy = d.normal(b, L, ch), d.normal(b, L, ch), d.normal(b, L, ch), -d.normal(ch).abs() - 0.1, d.normal(b, L, ch)
    want, _, states = ssd.ssd_gated_forward(x, r, i, A, want_states=True)
    grads = ssd.ssd_gated_backward(x, r, i, A, dy, states=states)
    for name, call in (("gated", lambda: ssd.ssd_gated_forward(x, r, i, A)[0]), ("gated_bwd", lambda: ssd.ssd_gated_backward(x, r, i, A, dy, states=states)["dx"])):
        lib.ssd_debug_set_wait_limit_ns(2_000_000)
        lib.ssd_debug_stall(1 << kinds[name])
        try:
            call()
            torch.cuda.synchronize()
            assert ssd.ssd_get_device_error() == _ffi.SSD_ERR_TIMEOUT
        finally:
            lib.ssd_debug_stall(0)
            lib.ssd_debug_set_wait_limit_ns(0)
        assert ssd.ssd_get_device_error() == 0
        assert torch.equal(call(), want if name == "gated" else grads["dx"])
    assert ssd.ssd_get_device_error() == 0


def test_the_same_bits_every_time(ssd):
    """Clusters of every size, and none: what the blocks of one give each other does not depend on who is first."""
    for b, L, ch, T in ((1, 9000, 128, torch.bfloat16), (2, 3000, 1088, torch.bfloat16), (2, 2100, 3200, torch.float32), (9, 700, 4096, torch.bfloat16)):
        d = Draw(21)
        x, r, i, dy = (d.normal(b, L, ch, dtype=T) for _ in range(4))
        A = -d.normal(ch).abs() - 0.01
        y, final, states = ssd.ssd_gated_forward(x, r, i, A, want_states=True)
        g = ssd.ssd_gated_backward(x, r, i, A, dy, states=states, want_dinit=True)
        for _ in range(15):
            y2, final2, states2 = ssd.ssd_gated_forward(x, r, i, A, want_states=True)
            g2 = ssd.ssd_gated_backward(x, r, i, A, dy, states=states, want_dinit=True)
            assert torch.equal(y, y2) and torch.equal(final, final2) and torch.equal(states, states2)
            assert all(torch.equal(g[k], g2[k]) for k in g)


def test_strides_and_pools_past_32_bits(ssd):
    """A batch stride, and a pool of states, of more than 2^31 elements."""
    d, T = Draw(22), torch.bfloat16
    big = torch.empty(2, (1 << 31) + 64, device="cuda", dtype=T)
    x = big[:, :40 * 32].unflatten(1, (40, 32))
    x.copy_(d.normal(2, 40, 32, dtype=T))
    A = -d.normal(32).abs() - 0.1
    y, _, _ = ssd.ssd_gated_forward(x, x, x, A)
    c = x.contiguous()
    assert torch.equal(y, ssd.ssd_gated_forward(c, c, c, A)[0])
    del big, x
    pool = torch.zeros((1 << 20) + 2, 2052, device="cuda")
    at = torch.tensor([(1 << 20) + 1, 5], dtype=torch.int32, device="cuda")
    v, A = d.normal(2, 2052), -d.normal(2052).abs() - 0.1
    small = torch.zeros(2, 2052, device="cuda")
    y, want = ssd.ssd_gated_step(v, v, v, A, pool, at), ssd.ssd_gated_step(v, v, v, A, small)
    assert torch.equal(y, want) and torch.equal(pool[at.long()], small) and float(pool.sum(dtype=torch.float64)) == float(small.sum(dtype=torch.float64))


def test_a_row_of_more_than_32_bits_of_elements(ssd):
    """The end of a row of 2^31 elements and more is the end of the same row cut short in front, from the state there."""
    d, L, ch, T = Draw(23), (1 << 19) + 200, 4104, torch.bfloat16
    x = d.normal(1, 1 << 12, ch, dtype=T).repeat(1, 129, 1)[:, :L]
    A = -d.normal(ch).abs() - 0.05
    y, final, states = ssd.ssd_gated_forward(x, x, x, A, want_states=True)
    start = L - L % 64 - 640
    part = x[:, start:].contiguous()
    want, wfinal, _ = ssd.ssd_gated_forward(part, part, part, A, states[:, start // 64].contiguous())
    # the runs are composed in another order: roundings of float32, then at most one of bfloat16 apart
    assert float((y[:, start:].float() - want.float()).abs().max()) <= 2.0 ** -7 * float(want.float().abs().max())
    assert float((final - wfinal).abs().max()) <= 1e-5 * float(wfinal.abs().max())
    g = ssd.ssd_gated_backward(x, x, x, A, y, states=states)
    tail = ssd.ssd_gated_backward(part, part, part, A, y[:, start:].contiguous(), states[:, start // 64].contiguous())
    for k in ("dx", "dr", "di"):
        assert float((g[k][:, start:].float() - tail[k].float()).abs().max()) <= 2.0 ** -7 * float(tail[k].float().abs().max()), k


def test_refusals(ssd):
    x, A = torch.zeros(2, 5, 16, device="cuda"), -torch.ones(16, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_gated_forward(x, x[..., :8], x, A)
    with pytest.raises(TypeError):
        ssd.ssd_gated_forward(x, x.half(), x, A)
    with pytest.raises(ValueError, match="shape"):
        ssd.ssd_gated_forward(x, x, x, A[:8])
    with pytest.raises(ValueError, match="dims"):
        ssd.ssd_gated_forward(x[0], x[0], x[0], A)
    with pytest.raises(ValueError, match="dense"):
        ssd.ssd_gated_forward(x, x, torch.zeros(2, 16, 5, device="cuda").transpose(1, 2), A)
    with pytest.raises(TypeError):
        ssd.ssd_gated_forward(x, x, x, A, lengths=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError, match="states"):
        ssd.ssd_gated_backward(x, x, x, A, x, states=torch.zeros(2, 2, 16, device="cuda"))
    with pytest.raises(ValueError, match="holds 1 rows"):
        ssd.ssd_gated_step(x[:, 0], x[:, 0], x[:, 0], A, torch.zeros(1, 16, device="cuda"))
    with pytest.raises(ssd.SSDError):
        ssd.ssd_gated_forward(x[:, :0], x[:, :0], x[:, :0], A)
