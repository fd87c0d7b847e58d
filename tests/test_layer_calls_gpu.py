"""How the layer operators are called: pieces from an iterator, other streams, graphs, flags and strides that a call does
not read.  (test_layer_gpu.py holds the values.)"""
import pytest
import torch

from test_layer_gpu import Draw, ssd  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("elsewhere", [False, True])
def test_conv_backward_takes_pieces_that_only_the_iterator_holds(ssd, elsewhere):  # noqa: F811
    """Each piece is made when it is asked for, and nothing but the call keeps it: its memory is not an output's."""
    d, b, L, pieces = Draw(21), 2, 64, [32, 16, 16]
    x, w, bias = d.normal(b, L, 64), d.normal(64, 4), d.normal(64)
    dy = tuple(d.normal(b, L, n) for n in pieces)
    want = ssd.ssd_conv_backward(x, w, bias, dy)
    stream = None
    if elsewhere:
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            made = [v.clone() for v in dy]  # the pieces belong to that stream
        got = ssd.ssd_conv_backward(x, w, bias, (made.pop(0) for _ in pieces), stream=stream)
        torch.cuda.current_stream().wait_stream(stream)
    else:
        got = ssd.ssd_conv_backward(x, w, bias, (v.clone() for v in dy))
    for name in ("dx", "dweight", "dbias"):
        assert torch.equal(got[name], want[name]), name


def test_a_slot_flag_waits_behind_a_range_flag(ssd):  # noqa: F811
    """Both raised before the first read: each is reported once."""
    d = Draw(9)
    x, bc = d.normal(1, 64, 4, 64, dtype=torch.bfloat16), d.normal(1, 64, 1, 64, dtype=torch.bfloat16)
    wide = bc.clone()
    wide[0, 3, 0, 5] = 1e6  # no float16
    ssd.ssd_forward(x, d.normal(1, 64, 4).abs(), -d.normal(4).abs(), wide, bc, None, None, 64)
    ssd.ssd_conv_step(d.normal(2, 8), d.normal(8, 4), None, d.normal(3, 3, 8), torch.tensor([3, 0], dtype=torch.int32, device="cuda"))
    assert [ssd.ssd_get_device_error() for _ in range(3)] == [7, 8, 0]


def test_strides_that_a_call_does_not_read(ssd):  # noqa: F811
    """A step's strides per token, and z's without a z, may hold anything."""
    import ctypes
    from state_space_sequence_ssd_gb300 import _ffi
    d, b, L, ch, N = Draw(31), 3, 5, 24, 16
    x, dt, B, C = d.normal(b, L, ch), d.normal(b, L, ch).abs(), d.normal(b, L, 1, N), d.normal(b, L, 1, N)
    A, state = -d.normal(ch, N).abs(), d.normal(b, ch, N)
    p = lambda t: t.data_ptr()  # noqa: E731
    lib, stream = _ffi.lib(), torch.cuda.current_stream().cuda_stream
    want = ssd.ssd_selective_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], None, state.clone())
    junk = _ffi.SelectiveStrides(L * ch, -1, L * ch, -3, -5, 7, L * N, 1, L * N, -2 ** 40)
    y = torch.empty(b, ch, device="cuda")
    assert lib.ssd_selective_step(_ffi.SSD_F32, p(x), p(dt), p(A), p(B), p(C), None, p(state), None, b, ctypes.addressof(junk), b,
                                  ch, 1, N, None, p(y), stream) == 0
    assert torch.equal(y, want)
    want, _ = ssd.ssd_selective_forward(x, dt, A, B, C)
    st = _ffi.SelectiveStrides(L * ch, ch, L * ch, ch, -1, -1, L * N, N, L * N, N)
    y = torch.empty(b, L, ch, device="cuda")
    assert lib.ssd_selective_forward(_ffi.SSD_F32, p(x), p(dt), p(A), p(B), p(C), None, None, None, ctypes.addressof(st), b, L, ch, 1,
                                     N, None, p(y), None, stream) == 0
    assert torch.equal(y, want)


def test_gradients_and_steps_on_another_stream(ssd):  # noqa: F811
    d, b, L, ch, N = Draw(61), 2, 70, 24, 16
    x, dt, B, C, dy = d.normal(b, L, ch), d.normal(b, L, ch).abs(), d.normal(b, L, 1, N), d.normal(b, L, 1, N), d.normal(b, L, ch)
    A, w, bias = -d.normal(ch, N).abs(), d.normal(ch, 4), d.normal(ch)
    _, mean, rstd = ssd.ssd_layer_norm_forward(x, bias)
    states, pool = d.normal(3, ch, N), d.normal(3, 3, ch)
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")

    def everything(**kw):
        s, p = states.clone(), pool.clone()
        if "stream" in kw:
            kw["stream"].wait_stream(torch.cuda.current_stream())
        out = [ssd.ssd_selective_backward(x, dt, A, B, C, bias, dy, **kw), ssd.ssd_conv_backward(x, w, bias, dy, **kw),
               ssd.ssd_conv_backward(x, w, bias, (dy[..., :16].contiguous(), dy[..., 16:].contiguous()), **kw),
               ssd.ssd_layer_norm_backward(x, bias, mean, rstd, dy, **kw),
               {"y": ssd.ssd_selective_step(x[:, 0], dt[:, 0], A, B[:, 0], C[:, 0], bias, s, slots, **kw), "state": s},
               {"y": ssd.ssd_conv_step(x[:, 0], w, bias, p, slots, **kw), "state": p}]
        if "stream" in kw:
            torch.cuda.current_stream().wait_stream(kw["stream"])
        return out

    want = everything()
    got = everything(stream=torch.cuda.Stream())
    for g, v in zip(got, want):
        for name in v:
            assert v[name] is None or torch.equal(g[name], v[name]), name


def test_a_decode_step_in_a_graph(ssd):  # noqa: F811
    """The steps and the norm of one token, captured once and replayed on new inputs with the states carried on."""
    d, b, ch, N = Draw(67), 4, 64, 16
    A, w, bias = -d.normal(ch, N).abs(), d.normal(ch, 4), d.normal(ch)
    slots = torch.tensor([5, -1, 0, 3], dtype=torch.int32, device="cuda")
    tokens = [(d.normal(b, ch), d.normal(b, ch).abs(), d.normal(b, 1, N), d.normal(b, 1, N)) for _ in range(5)]

    def step(x, dt, B, C, conv_state, state):
        h, _, _ = ssd.ssd_layer_norm_forward(x, bias)
        u = ssd.ssd_conv_step(h, w, bias, conv_state, slots)
        return ssd.ssd_selective_step(u, dt, A, B, C, bias, state, slots)

    states = lambda: (torch.ones(6, 3, ch, device="cuda"), torch.ones(6, ch, N, device="cuda"))  # noqa: E731
    plain = states()
    want = [step(*t, *plain) for t in tokens]
    held, inputs = states(), [v.clone() for v in tokens[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*inputs, *states())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(*inputs, *held)
    for s in held:
        s.fill_(1.0)
    for t, expected in zip(tokens, want):
        for to, v in zip(inputs, t):
            to.copy_(v)
        graph.replay()
        assert torch.equal(y, expected)
    assert all(torch.equal(a, b) for a, b in zip(held, plain))
