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
    # a token's decay enters a term of the state once, with its error and a rounding of its product and of its sum
    err = _walk(a, (e_a + 4 * U) * a * mag_before + (e_b + 4 * U) * bx.abs(), torch.zeros_like(h0))
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
    lam_err = back((after(e_a) + 6 * U) * after(a * lam_mag) + 2 * U * gy.abs(), torch.zeros_like(h0)) + 2 * U * lam_mag
    live = lambda val, e: (torch.where(keep, val, 0.0), torch.where(keep, e, 0.0))  # noqa: E731
    out = {"dx": live(lam * s * g, lam_err * s * g + lam_mag * s * g * (e_b + 2 * U))}
    # 1 - v and 1 - g are e^-r v and e^-i g: zero, with a relative error of one, below 2^-126
    e_vr, e_gr = (torch.where(q < LEAST, 1.0, e) for q, e in ((v_rest, e_v + r.abs() * U + 10 * U), (g_rest, e_g + i.abs() * U + 10 * U)))
    n = s * x.abs() * g * g_rest
    out["di"] = live(lam * s * x * g * g_rest, (lam_err + lam_mag * (e_b + e_gr + 4 * U)) * n)
    ratio = torch.where(w > 0, a * g / s.clamp(min=1e-300), 0.0)
    size = mag_before + ratio * x.abs()
    q = lam * u * a * (h_before - ratio * x)
    e_q = lam_err * u.abs() * a * size + lam_mag * u.abs() * a * (e_before + ratio * x.abs() * (e_a + e_b + 8 * U) + size * (e_u + e_a + 6 * U))
    out["dr"] = live(q * v_rest, (e_q + lam_mag * u.abs() * a * size * e_vr) * v_rest)
    q, e_q = live(q, e_q)
    # a thread adds a token in eight of each step's 64, then 8 warps, the blocks of a row and the rows
    terms = (lam_mag * u.abs() * a * size * keep).sum((0, 1))
    out["dA"] = (q.sum((0, 1)) / A, (e_q.sum((0, 1)) + terms * (L / 8 + 16 + 8 * b) * U) / A.abs())
    out["dinit"] = (a[:, 0] * lam[:, 0], a[:, 0] * (lam_err[:, 0] + lam_mag[:, 0] * (e_a[:, 0] + 2 * U)))
    return out
