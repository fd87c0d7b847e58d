"""layer_reference's definitions of the convolution and the selective scan on torch tensors in 64 bits, on any device, for sizes
that its numpy loops are too slow for (test_layer_sizes.py pins them to it).  ``mag=True`` as there."""
import torch
from torch.nn.functional import pad, softplus


def _kept(b, L, lengths, like):
    n = torch.full((b,), L, device=like.device) if lengths is None else lengths.long().clamp(0, L)
    return torch.arange(L, device=like.device)[None] < n[:, None], n


def conv(x, w, bias, init, lengths, silu, dy=None, dfinal=None, mag=False):
    """(y, final), or with dy: (dx, dweight, dbias, dinit)."""
    b, L, ch = x.shape
    W = w.shape[1]
    m = torch.abs if mag else (lambda v: v)
    init = x.new_zeros(b, W - 1, ch) if init is None else init
    bias = x.new_zeros(ch) if bias is None else bias
    keep, n = _kept(b, L, lengths, x)
    rows = torch.cat([init, torch.where(keep[..., None], x, 0.0)], 1)
    last = (n[:, None] + torch.arange(W - 1, device=x.device))[..., None].expand(-1, -1, ch)
    true = bias + sum(w[:, k] * rows[:, k:k + L] for k in range(W))
    pre = m(bias) + sum(m(w[:, k]) * m(rows[:, k:k + L]) for k in range(W))
    s = torch.sigmoid(true)
    if dy is None:
        y = pre * (s * (1 + true.abs() if mag else 1) if silu else 1)
        return torch.where(keep[..., None], y, 0.0), rows.gather(1, last)
    slope = s * (1 + true * (1 - s)) if silu else torch.ones_like(s)
    if mag and silu:
        slope = s * (1 + pre * (1 - s)) + pre
    g = torch.where(keep[..., None], m(dy) * m(slope), 0.0)
    wide = pad(g, (0, 0, W - 1, W - 1))
    drows = sum(m(w[:, k]) * wide[:, W - 1 - k:W - 1 - k + L + W - 1] for k in range(W))
    if dfinal is not None:
        drows = drows.scatter_add(1, last, m(dfinal))
    dw = torch.stack([(g * m(rows[:, k:k + L])).sum((0, 1)) for k in range(W)], 1)
    # what a row's own length leaves: its first tokens, and the states before them
    return torch.where(keep[..., None], drows[:, W - 1:], 0.0), dw, g.sum((0, 1)), drows[:, :W - 1]


def selective(x, dt, A, B, C, D, init, lengths, bias=None, soft=False, z=None, dy=None, dfinal=None, mag=False):
    """(y, final), or with dy a dict of gradients."""
    b, L, ch = x.shape
    G, N = B.shape[2:]
    m = torch.abs if mag else (lambda v: v)
    D = x.new_zeros(ch) if D is None else D
    h = x.new_zeros(b, ch, N) if init is None else m(init)
    keep, _ = _kept(b, L, lengths, x)
    clean = lambda v: torch.where(keep.reshape(b, L, *[1] * (v.dim() - 2)), v, 0.0)  # noqa: E731
    raw_dt = clean(dt) + (0.0 if bias is None else bias)
    d, slope = (softplus(raw_dt, threshold=1e9), torch.sigmoid(raw_dt)) if soft else (raw_dt, torch.ones_like(raw_dt))
    d, xs = clean(d), clean(x)
    Bs, Cs = (m(clean(v)).repeat_interleave(ch // G, 2) if G > 1 else m(clean(v)) for v in (B, C))
    gate, dgate = torch.ones_like(xs), None
    if z is not None:
        zz = clean(z)
        s = torch.sigmoid(zz)
        gate, dgate = zz * s, s * (1 + zz * (1 - s))
    hs, raw = [h], torch.zeros_like(xs)
    for t in range(L):
        h = torch.exp(d[:, t, :, None] * A) * h + (d[:, t] * m(xs[:, t]))[..., None] * Bs[:, t]
        if dy is not None:
            hs.append(h)
        raw[:, t] = (Cs[:, t] * h).sum(-1) + m(D) * m(xs[:, t])
    if dy is None:
        return clean(raw * m(gate)), h
    gy = clean(dy)
    g = m(gy) * m(gate)
    out = {k: torch.zeros_like(xs) for k in ("dx", "ddt")}
    if z is not None:
        out["dz"] = clean(m(gy) * raw * m(dgate))
    out["dA"], out["dB"], out["dC"] = torch.zeros_like(A), x.new_zeros(b, L, G, N), x.new_zeros(b, L, G, N)
    mu = x.new_zeros(b, ch, N) if dfinal is None else m(dfinal)
    for t in range(L - 1, -1, -1):
        lam = mu + Cs[:, t] * g[:, t, :, None]
        out["dB"][:, t] = (lam * (d[:, t] * m(xs[:, t]))[..., None]).reshape(b, G, ch // G, N).sum(2)
        out["dC"][:, t] = (hs[t + 1] * g[:, t, :, None]).reshape(b, G, ch // G, N).sum(2)
        byb = (lam * Bs[:, t]).sum(-1)
        mu = torch.exp(d[:, t, :, None] * A) * lam
        held = mu * hs[t]
        out["dA"] += (held * d[:, t, :, None]).sum(0)
        out["dx"][:, t] = byb * d[:, t] + m(D) * g[:, t]
        out["ddt"][:, t] = ((held * m(A)).sum(-1) + byb * m(xs[:, t])) * slope[:, t]
    for k in ("dx", "ddt", "dB", "dC"):
        out[k] = clean(out[k])
    out["dD"], out["ddt_bias"], out["dinit"] = (g * m(xs)).sum((0, 1)), out["ddt"].sum((0, 1)), mu
    return out
