"""The example model learns with the operators' gradients, and its decoding agrees with whole passes; and the convolution
with its pieces feeds the tensor-core scan, forward and backward."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_trains_and_decodes():
    spec = importlib.util.spec_from_file_location("selective_lm", os.path.join(ROOT, "examples", "selective_lm.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, off = example.main(steps=40, quiet=True)
    assert losses[0] > 3.5 and losses[-1] < 0.5 * losses[0], losses[::8]
    # float32 throughout: the two orders of summation differ by roundings only, logits are of order ten
    assert off < 1e-3


def test_conv_pieces_feed_the_tensor_core_scan():
    """One input projection's x, B and C through ssd_conv, then ssd_forward and ssd_backward, and back: every piece
    arrives where the scan's own layout wants it, and the gradient reaches the projection's columns."""
    import state_space_sequence_ssd_gb300 as ssd
    rand = torch.Generator(device="cuda")
    rand.manual_seed(1)
    b, L, H, P, G, N = 2, 160, 4, 64, 1, 64
    ch = H * P + 2 * G * N

    def normal(*shape):
        return torch.randn(shape, generator=rand, device="cuda")

    rows = normal(b, L, H * P + ch + H).to(torch.bfloat16)  # z | x B C | dt
    w, bias = normal(ch, 4) * 0.5, normal(ch) * 0.1
    xbc = rows[..., H * P:H * P + ch]
    (x, B, C), _ = ssd.ssd_conv_forward(xbc, w, bias, splits=[H * P, G * N, G * N])
    dt, A, D = torch.nn.functional.softplus(normal(b, L, H) - 4), -torch.exp(normal(H).abs()), normal(H)
    x4, B4, C4 = x.view(b, L, H, P), B.view(b, L, G, N), C.view(b, L, G, N)
    y, _ = ssd.ssd_forward(x4, dt, A, B4, C4, D, None, 64)
    dy = normal(b, L, H, P).to(torch.bfloat16)
    g = ssd.ssd_backward(x4, dt, A, B4, C4, D, None, dy, chunk_size=64)
    drows = torch.zeros_like(rows)
    pieces = (g["dx"].view(b, L, -1), g["dB"].view(b, L, -1), g["dC"].view(b, L, -1))
    out = ssd.ssd_conv_backward(xbc, w, bias, pieces, dx=drows[..., H * P:H * P + ch])
    assert ssd.ssd_get_device_error() == 0
    # the convolution by elementary operations, on the same pieces' gradients
    xf = xbc.float().requires_grad_()
    wide = torch.nn.functional.pad(xf, (0, 0, 3, 0))
    pre = sum(w[:, k] * wide[:, k:k + L] for k in range(4)) + bias
    act = pre * torch.sigmoid(pre)
    want, = torch.autograd.grad(act, xf, torch.cat([p.float() for p in pieces], -1))
    # both are float32 sums of four products of order |gradient|, rounded to bfloat16 here
    tol = 2.0 ** -8 * want.abs() + 1e-4 * want.abs().max()
    assert bool(((out["dx"].float() - want).abs() <= tol).all())
    assert bool((drows[..., :H * P] == 0).all()) and bool((drows[..., H * P + ch:] == 0).all())
    tol = 2.0 ** -8 * act.abs() + 1e-5
    assert bool(((torch.cat([x, B, C], -1).float() - act).abs() <= tol).all())
    assert bool(torch.isfinite(y.float()).all())
