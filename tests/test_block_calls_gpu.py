"""The gated recurrence, the grouped norm and the operators that were there in one layer: norm, short convolution, gated recurrence,
norm gated by z.  As a prompt and token by token, captured and replayed, and its gradients against the same layer in 64 bits."""
import pytest
import torch

from test_gated_gpu import TYPES, Draw, ssd  # noqa: F401

pytestmark = pytest.mark.gpu

CH, GROUPS, W = 96, 3, 4


def weights(d):
    return {"wn": 1 + d.normal(CH, scale=0.1), "bn": d.normal(CH, scale=0.1), "wc": d.normal(CH, W, scale=0.5), "bc": d.normal(CH, scale=0.1),
            "A": -d.normal(CH).abs() - 0.05, "wg": 1 + d.normal(CH, scale=0.1)}


def inputs(d, rows, T):
    """x, and the gates r, i and z as slices of one projection's rows."""
    gates = d.normal(*rows, 3 * CH, dtype=T)
    return d.normal(*rows, CH, dtype=T), gates[..., :CH], gates[..., CH:2 * CH], gates[..., 2 * CH:]


def prompt(ssd, w, x, r, i, z, lengths=None):  # noqa: F811
    h, mean, rstd = ssd.ssd_layer_norm_forward(x, w["wn"], w["bn"])
    u, conv = ssd.ssd_conv_forward(h, w["wc"], w["bc"], lengths=lengths)
    y, state, kept = ssd.ssd_gated_forward(u, r, i, w["A"], lengths=lengths, want_states=True)
    o, _, grstd = ssd.ssd_group_norm_forward(y, GROUPS, w["wg"], z=z, gate_first=True, rms=True)
    return o, conv, state, dict(h=h, mean=mean, rstd=rstd, u=u, y=y, kept=kept, grstd=grstd)


def token(ssd, w, x, r, i, z, conv, state, slots):  # noqa: F811
    h, _, _ = ssd.ssd_layer_norm_forward(x, w["wn"], w["bn"])
    u = ssd.ssd_conv_step(h, w["wc"], w["bc"], conv, slots)
    y = ssd.ssd_gated_step(u, r, i, w["A"], state, slots)
    return ssd.ssd_group_norm_forward(y, GROUPS, w["wg"], z=z, gate_first=True, rms=True)[0]


def layer64(w, x, r, i, z):
    """The layer from elementary operations, token by token."""
    f = torch.nn.functional
    h = f.layer_norm(x, (CH,), w["wn"], w["bn"])
    pad = f.pad(h, (0, 0, W - 1, 0))
    u = f.silu(w["bc"] + sum(w["wc"][:, k] * pad[:, k:k + x.shape[1]] for k in range(W)))
    a = torch.exp(w["A"] * torch.sigmoid(r))
    b = torch.sqrt(1 - a * a) * torch.sigmoid(i) * u
    s, ys = torch.zeros_like(b[:, 0]), []
    for t in range(x.shape[1]):
        s = a[:, t] * s + b[:, t]
        ys.append(s)
    q = (torch.stack(ys, 1) * f.silu(z)).unflatten(-1, (GROUPS, -1))
    return (q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-5)).flatten(-2) * w["wg"]


def test_a_prompt_and_its_last_tokens(ssd):  # noqa: F811
    d, b, L = Draw(1), 3, 150
    w = weights(d)
    x, r, i, z = inputs(d, (b, L), torch.float32)
    whole, conv, state, _ = prompt(ssd, w, x, r, i, z)
    want = layer64(*({k: v.double() for k, v in w.items()},), *(v.double() for v in (x, r, i, z)))
    # a dozen roundings of 2^-24 a token on values of order one, carried over the 20 tokens that the slowest channel keeps, through
    # norms whose slopes are of order one: 1e-5 is twenty times that
    assert float((whole.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())
    # the rows stop at lengths of their own and go on one by one, in slots of a pool
    lengths = torch.tensor([150, 0, 97], dtype=torch.int32, device="cuda")
    out, c, s, _ = prompt(ssd, w, x, r, i, z, lengths)
    pool_c, pool_s = torch.zeros(5, W - 1, CH, device="cuda"), torch.zeros(5, CH, device="cuda")
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    pool_c[slots.long()], pool_s[slots.long()] = c, s
    for step in range(3):
        at = (lengths.long() + step).clamp(max=L - 1)
        live = lengths + step < L
        pick = lambda v: v[torch.arange(b, device="cuda"), at]  # noqa: E731
        y = token(ssd, w, pick(x), pick(r), pick(i), pick(z), pool_c, pool_s, torch.where(live, slots, -1).to(torch.int32))
        assert float((y.double() - pick(want))[live].abs().max()) <= 1e-5 * float(want.abs().max())


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_a_token_in_a_graph(ssd, kind):  # noqa: F811
    d, b, T = Draw(2), 4, TYPES[kind]
    w = weights(d)
    tokens = [inputs(d, (b,), T) for _ in range(4)]
    slots = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device="cuda")
    states = lambda: (torch.ones(6, W - 1, CH, device="cuda", dtype=T), torch.ones(6, CH, device="cuda"))  # noqa: E731
    plain = states()
    want = [token(ssd, w, *t, *plain, slots) for t in tokens]
    held, ins = states(), [v.clone() for v in tokens[0]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        token(ssd, w, *ins, *states(), slots)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = token(ssd, w, *ins, *held, slots)
    for s in held:
        s.fill_(1.0)
    for t, expected in zip(tokens, want):
        for to, v in zip(ins, t):
            to.copy_(v)
        graph.replay()
        assert torch.equal(y, expected)
    assert all(torch.equal(p, q) for p, q in zip(held, plain))


def test_gradients_through_the_layer(ssd):  # noqa: F811
    d, b, L = Draw(3), 2, 140
    w = weights(d)
    x, r, i, z = inputs(d, (b, L), torch.float32)
    do = d.normal(b, L, CH)
    _, _, _, k = prompt(ssd, w, x, r, i, z)
    g = ssd.ssd_group_norm_backward(k["y"], GROUPS, w["wg"], None, None, k["grstd"], do, z=z, gate_first=True)
    s = ssd.ssd_gated_backward(k["u"], r, i, w["A"], g["dx"], states=k["kept"])
    c = ssd.ssd_conv_backward(k["h"], w["wc"], w["bc"], s["dx"])
    n = ssd.ssd_layer_norm_backward(x, w["wn"], k["mean"], k["rstd"], c["dx"])
    got = {"x": n["dx"], "r": s["dr"], "i": s["di"], "z": g["dz"], "wn": n["dweight"], "bn": n["dbias"], "wc": c["dweight"], "bc": c["dbias"],
           "A": s["dA"], "wg": g["dweight"]}
    leaf = {k2: v.double().requires_grad_() for k2, v in {**w, "x": x, "r": r, "i": i, "z": z}.items()}
    out = layer64(leaf, *(leaf[k2] for k2 in ("x", "r", "i", "z")))
    want = dict(zip(leaf, torch.autograd.grad(out, list(leaf.values()), do.double())))
    for name, value in want.items():
        # as above, through four operators; the sums over 280 tokens cancel by a factor of about 20
        assert float((got[name].double() - value).abs().max()) <= 5e-5 * float(value.abs().max()), name
