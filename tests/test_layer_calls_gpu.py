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
