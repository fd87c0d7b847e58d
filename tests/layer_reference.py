"""The layer operators' definitions in 64 bits, token by token (numpy), and the scale of their rounding errors.

Every function takes float64 arrays.  With ``mag=True`` the same sums are formed from the magnitudes of their
terms (decays, which are positive, stay as they are): the result S of that bounds the error of a float32
evaluation, which is at most (number of roundings on a term's way) * (rounding) * S.
"""
import numpy as np


def sigmoid(v):
    return 0.5 * (1 + np.tanh(0.5 * v))


def softplus(v):
    return np.maximum(v, 0) + np.log1p(np.exp(-np.abs(v)))


def conv(x, w, bias, init, lengths, silu, dy=None, dfinal=None, mag=False):
    """(y, final), or with dy: (dx, dweight, dbias, dinit)."""
    b, L, ch = x.shape
    W = w.shape[1]
    m = np.abs if mag else (lambda v: v)
    init = np.zeros((b, W - 1, ch)) if init is None else init
    bias = np.zeros(ch) if bias is None else bias
    y, final = np.zeros((b, L, ch)), np.zeros((b, W - 1, ch))
    dx, dw, db, dinit = np.zeros((b, L, ch)), np.zeros((ch, W)), np.zeros(ch), np.zeros((b, W - 1, ch))
    for i in range(b):
        n = L if lengths is None else min(max(int(lengths[i]), 0), L)
        rows = np.concatenate([init[i], x[i, :n]])
        final[i] = rows[n:]
        drows = np.zeros_like(rows)
        if dfinal is not None:
            drows[n:] += m(dfinal[i])
        for t in range(n):
            true = bias + sum(w[:, k] * rows[t + k] for k in range(W))
            pre = m(bias) + sum(m(w[:, k]) * m(rows[t + k]) for k in range(W))
            s = sigmoid(true)
            y[i, t] = pre * (s * (1 + (np.abs(true) if mag else 0)) if silu else 1)
            if dy is None:
                continue
            slope = s * (1 + true * (1 - s)) if silu else np.ones(ch)
            if mag and silu:  # the error of pre moves the slope too
                slope = s * (1 + pre * (1 - s)) + pre
            g = m(dy[i, t]) * m(slope)
            db += g
            for k in range(W):
                dw[:, k] += g * m(rows[t + k])
                drows[t + k] += g * m(w[:, k])
        dinit[i], dx[i, :n] = drows[:W - 1], drows[W - 1:]
    return (y, final) if dy is None else (dx, dw, db, dinit)


def effective_dt(dt, bias, soft, limit):
    v = dt if bias is None else dt + bias
    raw = v
    v = softplus(v) if soft else v
    slope = sigmoid(raw) if soft else np.ones_like(v)
    if limit is not None:
        slope = np.where((v >= limit[0]) & (v <= limit[1]), slope, 0.0)
        v = np.clip(v, *limit)
    return v, slope


def selective(x, dt, A, B, C, D, init, lengths, bias=None, soft=False, limit=None, z=None, dy=None, dfinal=None, mag=False):
    """(y, final), or with dy a dict of gradients."""
    b, L, ch = x.shape
    G, N = B.shape[2:]
    m = np.abs if mag else (lambda v: v)
    D = np.zeros(ch) if D is None else D
    h = np.zeros((b, ch, N)) if init is None else m(init).astype(np.float64)
    n = np.full(b, L) if lengths is None else np.clip(lengths, 0, L)
    keep = np.arange(L)[None] < n[:, None]
    clean = lambda v: np.where(keep.reshape(b, L, *[1] * (v.ndim - 2)), v, 0.0)  # noqa: E731
    d, slope = effective_dt(clean(dt), bias, soft, limit)
    d, xs, Bs, Cs = clean(d), clean(x), m(clean(B)).repeat(ch // G, 2), m(clean(C)).repeat(ch // G, 2)
    gate, dgate = np.ones_like(xs), np.zeros_like(xs)
    if z is not None:
        zz = clean(z)
        s = sigmoid(zz)
        gate, dgate = zz * s, s * (1 + zz * (1 - s))
    hs, raw = [h], np.zeros((b, L, ch))
    for t in range(L):
        h = np.exp(d[:, t, :, None] * A) * h + (d[:, t] * m(xs[:, t]))[..., None] * Bs[:, t]
        hs.append(h)
        raw[:, t] = (Cs[:, t] * h).sum(-1) + m(D) * m(xs[:, t])
    if dy is None:
        return clean(raw * m(gate)), h
    gy = clean(dy)
    g = m(gy) * m(gate)
    out = {k: np.zeros_like(xs) for k in ("dx", "ddt")}
    out["dz"] = clean(m(gy) * raw * m(dgate))
    out["dA"], out["dB"], out["dC"] = np.zeros((ch, N)), np.zeros((b, L, G, N)), np.zeros((b, L, G, N))
    mu = np.zeros((b, ch, N)) if dfinal is None else m(dfinal).astype(np.float64)
    for t in range(L - 1, -1, -1):
        lam = mu + Cs[:, t] * g[:, t, :, None]
        a = np.exp(d[:, t, :, None] * A)
        out["dB"][:, t] = (lam * (d[:, t] * m(xs[:, t]))[..., None]).reshape(b, G, ch // G, N).sum(2)
        out["dC"][:, t] = (hs[t + 1] * g[:, t, :, None]).reshape(b, G, ch // G, N).sum(2)
        byb = (lam * Bs[:, t]).sum(-1)
        mu = a * lam
        held = mu * hs[t]
        out["dA"] += (held * d[:, t, :, None]).sum(0)
        out["dx"][:, t] = byb * d[:, t] + m(D) * g[:, t]
        out["ddt"][:, t] = ((held * m(A)).sum(-1) + byb * m(xs[:, t])) * slope[:, t]
    for k in ("dx", "ddt", "dB", "dC"):
        out[k] = clean(out[k])
    out["dD"], out["ddt_bias"], out["dinit"] = (g * m(xs)).sum((0, 1)), out["ddt"].sum((0, 1)), mu
    return out


def norm(x, w, bias, eps, dy=None, mag=False):
    """(y, mean, rstd), or with dy (dx, dweight, dbias)."""
    m = np.abs if mag else (lambda v: v)
    mean = x.mean(-1, keepdims=True)
    rstd = 1 / np.sqrt(((x - mean) ** 2).mean(-1, keepdims=True) + eps)
    # the mean's own rounding is relative to the mean of magnitudes
    xhat = (np.abs(x) + np.abs(x).mean(-1, keepdims=True)) * rstd if mag else (x - mean) * rstd
    w = np.ones(x.shape[-1]) if w is None else w
    bias = np.zeros(x.shape[-1]) if bias is None else bias
    if dy is None:
        return xhat * m(w) + m(bias), mean[:, 0], rstd[:, 0]
    g = m(dy) * m(w)
    s1, s2 = g.mean(-1, keepdims=True), (g * xhat).mean(-1, keepdims=True)
    dx = rstd * (g + s1 + xhat * s2) if mag else rstd * (g - s1 - xhat * s2)
    return dx, (m(dy) * xhat).sum(0), m(dy).sum(0)
