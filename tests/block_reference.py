"""The definitions of the gated recurrence, the grouped norm and the rotary positions on torch tensors in 64 bits, on any device,
each with a bound of what a float32 evaluation of it may be off by.

Bounds.  U = 2^-24 is a float32 rounding.  The special function unit's exponential, reciprocal, root and reciprocal root are within
4 U of the value for the argument that they get; an exponential's argument is rounded too, which moves it by |argument| U.  A
value's relative error is the sum of those of its factors; a sum's error the sum of its terms' errors and a rounding of the magnitude
of its terms for every addition on a term's way.
"""
import torch

U = 2.0 ** -24
SPAN = 64
LEAST = 2.0 ** -125  # below 2^-126 a gate and 1 - a^2 are zero


def kept(b, L, lengths, like):
    """(batch, L, 1): whether a position is within its row's length."""
    n = torch.full((b,), L, device=like.device) if lengths is None else lengths.long().clamp(0, L)
    return (torch.arange(L, device=like.device)[None] < n[:, None])[..., None]


def _walk(a, b, h):
    """h after every token of h <- a h + b."""
    out = []
    for t in range(b.shape[1]):
        h = a[:, t] * h + b[:, t]
        out.append(h)
    return torch.stack(out, 1)


def _before(h, first):
    return torch.cat([first[:, None], h[:, :-1]], 1)


def gated(x, r, i, A, init=None, lengths=None, dy=None, dfinal=None):
    """{name: (value, bound)} of y, final and states, or with dy of the gradients."""
    b, L, ch = x.shape
    keep = kept(b, L, lengths, x)
    x, r, i = (torch.where(keep, v, 0.0) for v in (x, r, i))
    h0 = x.new_zeros(b, ch) if init is None else init
    v, g, v_rest, g_rest = torch.sigmoid(r), torch.sigmoid(i), torch.sigmoid(-r), torch.sigmoid(-i)
    # the exponential, its argument, the sum, the product of both denominators, its reciprocal, the product with the other's
    e_v, e_g = (12 + r.abs()) * U, (12 + i.abs()) * U
    e_v, e_g = (torch.where(q < LEAST, 1.0, e) for q, e in ((v, e_v), (g, e_g)))
    u = torch.where(keep, A * v, 0.0)
    a = torch.exp(u)
    w = -torch.expm1(2 * u)
    s = torch.sqrt(w)
    far = u <= -0.25
    e_u = e_v + U
    e_a = u.abs() * (e_u + U) + U + torch.where(far, 4 * U, 0.0)
    # near zero the polynomial's ten roundings and the two of w; far from it a's error over what 1 - a leaves
    e_s = (e_u + 12 * U + torch.where(far, 4 * a * e_a / w.clamp(min=0.3), 0.0)) / 2 + 6 * U
    # where v or 1 - a^2 is taken as zero so is s, and its relative error is one
    e_s = torch.where((w < LEAST) | (v < LEAST), 1.0, e_s)
    bx = s * g * x
    e_b = e_s + e_g + 3 * U
    h = _walk(a, bx, h0)
    mag = _walk(a, bx.abs(), h0.abs())
    mag_before, h_before = _before(mag, h0.abs()), _before(h, h0)
    # a decay below 2^-126 is taken as that
    off_a = e_a * a + torch.where(u < -86, LEAST, 0.0)
    # a token's decay enters a term of the state once, with its error and a rounding of its product and of its sum
    err = _walk(a, (off_a + 4 * U * a) * mag_before + (e_b + 4 * U) * bx.abs(), torch.zeros_like(h0))
    if dy is None:
        at = torch.arange(0, L, SPAN, device=x.device)
        return {"y": tuple(torch.where(keep, q, 0.0) for q in (h, err)), "final": (h[:, -1], err[:, -1]),
                "states": (h_before[:, at], _before(err, torch.zeros_like(h0))[:, at])}
    e_before = _before(err, torch.zeros_like(h0)) + 4 * U * mag_before
    gy = torch.where(keep, dy, 0.0)
    last = torch.zeros_like(h0) if dfinal is None else dfinal
    back = lambda q, first: _walk(_before(a.flip(1), torch.ones_like(h0)), q.flip(1), first).flip(1)  # noqa: E731
    lam, lam_mag = back(gy, last), back(gy.abs(), last.abs())
    after = lambda q: torch.cat([q[:, 1:], torch.zeros_like(q[:, :1])], 1)  # noqa: E731
    lam_err = back(after((off_a + 6 * U * a) * lam_mag) + 2 * U * gy.abs(), torch.zeros_like(h0)) + 2 * U * lam_mag
    live = lambda val, e: (torch.where(keep, val, 0.0), torch.where(keep, e, 0.0))  # noqa: E731
    out = {"dx": live(lam * s * g, lam_err * s * g + lam_mag * s * g * (e_b + 2 * U))}
    # 1 - v and 1 - g are e^-r v and e^-i g: zero, with a relative error of one, below 2^-126
    e_vr, e_gr = (torch.where(q < LEAST, 1.0, e) for q, e in ((v_rest, e_v + r.abs() * U + 10 * U), (g_rest, e_g + i.abs() * U + 10 * U)))
    n = s * x.abs() * g * g_rest
    out["di"] = live(lam * s * x * g * g_rest, (lam_err + lam_mag * (e_b + e_gr + 4 * U)) * n)
    per_s = torch.where(w > 0, g / s.clamp(min=1e-300), 0.0)
    ratio = a * per_s
    size = mag_before + ratio * x.abs()
    q = lam * u * a * (h_before - ratio * x)
    e_size = e_before + (per_s * off_a + ratio * (e_b + 8 * U)) * x.abs() + size * (e_u + 6 * U)
    e_q = lam_err * u.abs() * a * size + lam_mag * u.abs() * (off_a * size + (a + off_a) * e_size)
    out["dr"] = live(q * v_rest, (e_q + lam_mag * u.abs() * a * size * e_vr) * v_rest)
    q, e_q = live(q, e_q)
    # a thread adds a token in eight of each step's 64, then 8 warps, the blocks of a row and the rows
    terms = (lam_mag * u.abs() * a * size * keep).sum((0, 1))
    out["dA"] = (q.sum((0, 1)) / A, (e_q.sum((0, 1)) + terms * (L / 8 + 16 + 8 * b) * U) / A.abs())
    out["dinit"] = (a[:, 0] * lam[:, 0], a[:, 0] * (lam_err[:, 0] + lam_mag[:, 0] * 2 * U) + off_a[:, 0] * lam_mag[:, 0])
    return out


def _silu(v):
    """silu and its slope, each with the bound of its error."""
    s = torch.sigmoid(v)
    slope = s * (1 + v * (1 - s))
    return s, v * s, (v * s).abs() * (12 + v.abs()) * U, slope, s * (1 + v.abs() * (1 - s)) * (30 + 2 * v.abs()) * U


def group_norm(x, groups, weight=None, bias=None, z=None, gate_first=False, silu=False, rms=False, eps=1e-5, stats=None, dy=None):
    """{name: (value, bound)} of y, mean and rstd; with stats (mean, rstd), which are taken as they are, and dy of the gradients."""
    rows, width = x.shape
    per = width // groups
    # a thread adds at most 32 values, or one in 256 of a wide group's; then the threads' sums
    k = (per / 256 + 60) * U
    split = lambda t: t.unflatten(-1, (groups, per))  # noqa: E731
    w = torch.ones_like(x[0]) if weight is None else weight
    b = torch.zeros_like(w) if bias is None else bias
    if z is not None:
        sz, gz, e_gz, slope_z, e_slope_z = _silu(z)
    q, e_q = (x * gz, x.abs() * e_gz + (x * gz).abs() * 2 * U) if gate_first else (x, torch.zeros_like(x))
    q, e_q = split(q), split(e_q)
    if stats is None:
        mean = q.mean(-1, keepdim=True) * (not rms)
        e_mean = (q.abs().mean(-1, keepdim=True) * k + e_q.mean(-1, keepdim=True)) * (not rms)
        off = q - mean
        e_off = e_q + e_mean + off.abs() * U
        var = off.square().mean(-1, keepdim=True)
        rstd = 1 / torch.sqrt(var + eps)
        e_rstd = (off.abs() * e_off).mean(-1, keepdim=True) / (var + eps) + (k + 8 * U)
        n = (off * rstd).flatten(1) * w
        e_n = (e_off * rstd + (off * rstd).abs() * (e_rstd + 4 * U)).flatten(1) * w.abs() + 2 * U * (n.abs() + b.abs())
        n = n + b
        if silu:
            _, y, e_y, *_ = _silu(n)
            e_y = e_y + 1.1 * e_n
        elif z is not None and not gate_first:
            y, e_y = n * gz, e_n * gz.abs() + n.abs() * (e_gz + 2 * U * gz.abs())
        else:
            y, e_y = n, e_n
        return {"y": (y, e_y), "mean": (mean[..., 0], e_mean[..., 0]), "rstd": (rstd[..., 0], (rstd * e_rstd)[..., 0])}
    mean, rstd = (torch.zeros_like(q[..., :1]) if v is None else v[..., None] for v in stats)
    xh = ((q - mean) * rstd).flatten(1)
    e_xh = (e_q * rstd + (q.abs() + mean.abs()) * rstd * 4 * U).flatten(1)
    n, e_n = xh * w + b, e_xh * w.abs() + 2 * U * (xh * w).abs() + U * b.abs()
    out, g, e_g = {}, dy, torch.zeros_like(dy)
    if silu:
        _, _, _, slope, e_slope = _silu(n)
        g, e_g = dy * slope, dy.abs() * (e_slope + 0.6 * e_n + U)  # the slope's own slope is at most 0.5
    if z is not None and not gate_first:
        out["dz"] = dy * n * slope_z, dy.abs() * (e_n * slope_z.abs() + n.abs() * (e_slope_z + 3 * U * slope_z.abs()))
        g, e_g = dy * gz, dy.abs() * (e_gz + 2 * U * gz.abs())
    gw, e_gw, xs, e_xs = split(g * w), split(e_g * w.abs() + U * (g * w).abs()), split(xh), split(e_xh)
    s1, m1 = gw.mean(-1, keepdim=True) * (not rms), gw.abs().mean(-1, keepdim=True) * (not rms)
    s2, m2 = (gw * xs).mean(-1, keepdim=True), (gw * xs).abs().mean(-1, keepdim=True)
    e_s1 = m1 * k + e_gw.mean(-1, keepdim=True) * (not rms)
    e_s2 = m2 * k + (e_gw * xs.abs() + gw.abs() * e_xs).mean(-1, keepdim=True)
    dq = (rstd * (gw - s1 - xs * s2)).flatten(1)
    e_dq = (rstd * (e_gw + e_s1 + xs.abs() * e_s2 + e_xs * s2.abs() + 6 * U * (gw.abs() + m1 + xs.abs() * m2))).flatten(1)
    if gate_first:
        out["dz"] = dq * x * slope_z, x.abs() * (e_dq * slope_z.abs() + dq.abs() * (e_slope_z + 3 * U * slope_z.abs()))
        dq, e_dq = dq * gz, e_dq * gz.abs() + dq.abs() * (e_gz + 2 * U * gz.abs())
    out["dx"] = dq, e_dq
    # a block adds its rows, up to 256 of them at once, then 32 sums of the blocks' rows
    terms = (rows / 300 + 320) * U
    out["dweight"] = (g * xh).sum(0), (e_g * xh.abs() + g.abs() * e_xh).sum(0) + (g * xh).abs().sum(0) * terms
    out["dbias"] = g.sum(0), e_g.sum(0) + g.abs().sum(0) * terms
    return out


def rotary(x, frequencies, positions=None, lengths=None, interleaved=False, scale=1.0, inverse=False, fast=False):
    """(value, bound) of x (batch, L, heads, dim) turned; fast: the sines of 16-bit tensors."""
    b, L = x.shape[:2]
    at = torch.arange(L, device=x.device).expand(b, L)
    if positions is not None:
        at = positions.long() if positions.dim() == 2 else at + positions.long()[:, None]
    angle = at[..., None, None].double() * frequencies
    cos, sin = scale * torch.cos(angle), scale * torch.sin(angle) * (-1 if inverse else 1)
    n = 2 * len(frequencies)
    one, two = (slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n))
    y, bound = x.clone(), torch.zeros_like(x)
    p, q = x[..., one], x[..., two]
    y[..., one], y[..., two] = p * cos - q * sin, p * sin + q * cos
    # the angle to 2^-32 of a turn and a float32 rounding of it, the functions' error, the products and their sum
    e = (2.0 ** -19 if fast else 14 * U) * abs(scale) + 3 * U * abs(scale)
    bound[..., one] = bound[..., two] = (p.abs() + q.abs()) * e
    keep = kept(b, L, lengths, x)[..., None]
    return torch.where(keep, y, 0.0), torch.where(keep, bound, 0.0)
