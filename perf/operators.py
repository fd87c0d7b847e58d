"""The cases that the layer operators around the scan are measured on, with their plain forms.

Three operators, each for prompts or training rows, for its gradient, and (two of them) for single tokens:

  conv_*       the short causal depthwise convolution in front of a scan: `width` taps per channel, a bias,
               silu, the last width - 1 inputs as its state, its output in up to three dense pieces
               (x, B and C of a scan);
  selective_*  the selective scan with one decay per channel and state entry and one dt per channel;
  norm_*       the layer norm in front of a layer, and the reduction of its weight's gradient.

`run` makes the library's calls where `own` is true, and computes the same from elementary torch
operations in 32 bits, rounded once at the end, where it is false.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a short prompt of a small layer: 4 heads of 64, state size 64, one group (latency counts)
        dict(name="conv_prompt_short", op="conv_forward", dtype="bf16", batch=1, seqlen=512, pieces="256,64,64", width=4,
             bias=True, silu=True, offset=256, tail=4, init=True, ragged=False),
        # a layer's prompt or training forward: 64 heads of 64, state size 128; the channels are a slice of the
        # input projection's rows (z | x B C | dt)
        dict(name="conv_prompt", op="conv_forward", dtype="bf16", batch=2, seqlen=4096, pieces="4096,128,128", width=4,
             bias=True, silu=True, offset=4096, tail=64, init=False, ragged=False),
        # the gradient at the same layer: dx in 16 bits and dB, dC in 32, as the scan's backward pass returns them
        dict(name="conv_grad", op="conv_backward", dtype="bf16", batch=2, seqlen=4096, pieces="4096,128,128", width=4,
             bias=True, silu=True, offset=4096, tail=64, init=False, ragged=False),
        # one token of 256 sequences, their states in slots of a pool, a few rows of the batch idle
        dict(name="conv_decode", op="conv_step", dtype="bf16", batch=256, pieces="4096,128,128", width=4, bias=True, silu=True,
             offset=4096, tail=64, slots=True),
        # a short prompt in 32 bits, its state carried in (latency counts)
        dict(name="selective_prompt_short", op="selective_forward", dtype="f32", batch=1, seqlen=512, channels=256, ngroups=1,
             dstate=16, gate=True, softplus=True, init=True, ragged=False, rank=16),
        # a layer's prompt or training forward
        dict(name="selective_prompt", op="selective_forward", dtype="bf16", batch=2, seqlen=4096, channels=4096, ngroups=1,
             dstate=16, gate=True, softplus=True, init=False, ragged=False, rank=128),
        # prompts of unlike lengths padded to one row length, one of them empty; odd sizes, two groups
        dict(name="selective_ragged", op="selective_forward", dtype="f16", batch=5, seqlen=1777, channels=1530, ngroups=2,
             dstate=13, gate=False, softplus=True, init=True, ragged=True, rank=48),
        # one long document
        dict(name="selective_long", op="selective_forward", dtype="bf16", batch=1, seqlen=65536, channels=2048, ngroups=1,
             dstate=16, gate=True, softplus=True, init=True, ragged=False, rank=64),
        # the gradient of a training step
        dict(name="selective_grad", op="selective_backward", dtype="bf16", batch=2, seqlen=4096, channels=2048, ngroups=1,
             dstate=16, gate=True, softplus=True, init=False, ragged=False, rank=64),
        # one token of 256 sequences
        dict(name="selective_decode", op="selective_step", dtype="bf16", batch=256, channels=4096, ngroups=1, dstate=16, gate=True,
             softplus=True, slots=True, rank=128),
        # the norm in front of a layer, and its gradient with the weight's and the bias's
        dict(name="norm_prompt", op="norm_forward", dtype="bf16", rows=8192, width=2048, bias=True, tail=0),
        dict(name="norm_grad", op="norm_backward", dtype="bf16", rows=8192, width=2048, bias=True, tail=0),
    ]


def _size(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm; half of them are a multiple of 8."""
    n = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return max(lo, min(hi, (n + 4) // 8 * 8)) if n > 16 and rng.random() < 0.5 else n


def draw(rng):
    cap = work(listed()[7])
    while True:
        case = _draw(rng)
        w = work(case)
        if w["bytes"] <= cap["bytes"] / 2 and w["flops"] <= cap["flops"] / 2:
            return case


def _draw(rng):
    op = rng.choice(["conv_forward", "conv_backward", "conv_step", "selective_forward", "selective_forward",
                     "selective_backward", "selective_step", "norm_forward", "norm_backward"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("conv"):
        n0 = _size(rng, 64, 8192)
        pieces = [n0] if coin() else [n0, *(2 * [rng.choice([16, 64, 128, 256])])]
        case.update(pieces=",".join(map(str, pieces)), width=rng.choice([2, 3, 4, 4]), bias=coin(), silu=rng.random() < 0.8,
                    offset=rng.choice([0, n0, 24]), tail=rng.choice([0, 8, 64, 3]))
        if op == "conv_step":
            case.update(batch=_size(rng, 1, 512), slots=coin())
        else:
            case.update(batch=rng.choice([1, 2, 3, 8]), seqlen=_size(rng, 1, 32768), init=coin(), ragged=coin())
    elif op.startswith("selective"):
        groups = rng.choice([1, 1, 2, 4])
        case.update(channels=groups * _size(rng, 64, 8192 // groups), ngroups=groups, dstate=rng.choice([8, 16, 16, 16, 13, 32, 64]),
                    gate=coin(), softplus=rng.random() < 0.8, rank=rng.choice([0, 16, 48, 128]))
        if op == "selective_step":
            case.update(batch=_size(rng, 1, 512), slots=coin())
        else:
            case.update(batch=rng.choice([1, 2, 3, 8]), seqlen=_size(rng, 1, 32768 if op == "selective_forward" else 8192), init=coin(),
                        ragged=coin())
    else:
        case.update(rows=_size(rng, 1, 65536), width=_size(rng, 64, 16384), bias=coin(), tail=rng.choice([0, 0, 64, 3]))
    return case


# ------------------------------------------------------------------------------------------------ inputs


def _lengths(case, rand):
    """Row lengths from nothing to the whole row, or None."""
    if not case["ragged"]:
        return None
    n = (torch.rand(case["batch"], generator=rand, device="cuda") * (case["seqlen"] + 1)).to(torch.int32)
    n[0] = case["seqlen"]
    n[1:2] = 0
    return n


def _slots(case, rand):
    """Each row's place in a pool eight larger than the batch; one row in sixteen is idle (-1)."""
    if not case["slots"]:
        return case["batch"], None
    pool = case["batch"] + 8
    s = torch.randperm(pool, generator=rand, device="cuda")[: case["batch"]].to(torch.int32)
    s[torch.rand(case["batch"], generator=rand, device="cuda") < 1 / 16] = -1
    return pool, s


def prepare(case, seed):
    rand = torch.Generator(device="cuda")
    rand.manual_seed(seed)
    T, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, dtype=T, scale=1.0):
        return (torch.randn(shape, generator=rand, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=rand, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if op.startswith("conv"):
        pieces, W = [int(n) for n in case["pieces"].split(",")], case["width"]
        ch = sum(pieces)
        rows = (case["batch"],) if op == "conv_step" else (case["batch"], case["seqlen"])
        # the channels are columns of a projection's rows
        s.update(x=normal(*rows, case["offset"] + ch + case["tail"])[..., case["offset"]:case["offset"] + ch], pieces=pieces,
                 weight=uniform(ch, W, lo=-W ** -0.5, hi=W ** -0.5), bias=uniform(ch, lo=-0.5, hi=0.5) if case["bias"] else None)
        if op == "conv_step":
            pool, s["slots"] = _slots(case, rand)
            s["state"] = normal(pool, W - 1, ch)
        else:
            s.update(init=normal(case["batch"], W - 1, ch) if case["init"] else None, lengths=_lengths(case, rand))
        if op == "conv_backward":
            s["dy"] = [normal(*rows, n, dtype=T if i == 0 else torch.float32) for i, n in enumerate(pieces)]
            s["dfinal"] = normal(case["batch"], W - 1, ch) if case["init"] else None
    elif op.startswith("selective"):
        ch, G, N, R = case["channels"], case["ngroups"], case["dstate"], case["rank"]
        rows = (case["batch"],) if op == "selective_step" else (case["batch"], case["seqlen"])
        # x from the convolution; z a slice of the input projection, B and C slices of one that also gives dt's low rank
        dbc = normal(*rows, R + 2 * G * N)
        # dt in [0.001, 0.1] around its bias, as such layers are initialised
        start = torch.exp(uniform(ch, lo=math.log(0.001), hi=math.log(0.1)))
        soft = case["softplus"]
        s.update(x=torch.nn.functional.silu(normal(*rows, ch)), B=dbc[..., R:R + G * N].unflatten(-1, (G, N)),
                 dt=normal(*rows, ch, scale=0.5) if soft else uniform(*rows, ch, lo=0.001, hi=0.1).to(T),
                 C=dbc[..., R + G * N:].unflatten(-1, (G, N)), z=normal(*rows, 2 * ch)[..., ch:] if case["gate"] else None,
                 A=-torch.arange(1, N + 1, device="cuda") * torch.exp(normal(ch, N, dtype=torch.float32, scale=0.1)),
                 D=1 + normal(ch, dtype=torch.float32, scale=0.1), bias=torch.log(torch.expm1(start)) if soft else None)
        if op == "selective_step":
            pool, s["slots"] = _slots(case, rand)
            s["state"] = normal(pool, ch, N, dtype=torch.float32, scale=0.3)
        else:
            s.update(init=normal(case["batch"], ch, N, dtype=torch.float32, scale=0.3) if case["init"] else None,
                     lengths=_lengths(case, rand))
        if op == "selective_backward":
            s.update(dy=normal(*rows, ch), dfinal=normal(case["batch"], ch, N, dtype=torch.float32) if case["init"] else None)
    else:
        n, w = case["rows"], case["width"]
        # a residual stream: channels of unlike scale around unlike means
        x = normal(n, w + case["tail"], dtype=torch.float32) * torch.exp(normal(w + case["tail"], dtype=torch.float32, scale=0.5))
        s.update(x=(x + normal(n, 1, dtype=torch.float32)).to(T)[:, :w], weight=1 + normal(w, dtype=torch.float32, scale=0.1),
                 bias=normal(w, dtype=torch.float32, scale=0.1) if case["bias"] else None, eps=1e-5)
        if op == "norm_backward":
            xf = s["x"].float()
            s["mean"] = xf.mean(-1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(-1) + s["eps"])
            s["dy"] = normal(n, w)
    return s


# ------------------------------------------------------------------------------------------------ the passes


def run(s):
    return _library(s) if own else PLAIN[s["case"]["op"]](s)


def _library(s):
    import state_space_sequence_ssd_gb300 as ssd
    c, op = s["case"], s["case"]["op"]
    if op == "conv_forward":
        y, final = ssd.ssd_conv_forward(s["x"], s["weight"], s["bias"], s["init"], s["lengths"], silu=c["silu"], splits=s["pieces"])
        return {"y": y, "final": final}
    if op == "conv_backward":
        return ssd.ssd_conv_backward(s["x"], s["weight"], s["bias"], s["dy"], s["init"], s["lengths"], silu=c["silu"],
                                     dfinal=s["dfinal"], want_dinit=c["init"])
    if op == "conv_step":
        y = ssd.ssd_conv_step(s["x"], s["weight"], s["bias"], s["state"], s["slots"], silu=c["silu"], splits=s["pieces"])
        return {"y": y, "state": s["state"]}
    if op == "selective_forward":
        y, final = ssd.ssd_selective_forward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["init"], s["lengths"],
                                             dt_bias=s["bias"], dt_softplus=c["softplus"], z=s["z"])
        return {"y": y, "final": final}
    if op == "selective_backward":
        return ssd.ssd_selective_backward(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["dy"], s["init"], s["lengths"],
                                          dt_bias=s["bias"], dt_softplus=c["softplus"], z=s["z"], dfinal=s["dfinal"],
                                          want_dinit=c["init"])
    if op == "selective_step":
        y = ssd.ssd_selective_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["D"], s["state"], s["slots"],
                                   dt_bias=s["bias"], dt_softplus=c["softplus"], z=s["z"])
        return {"y": y, "state": s["state"]}
    if op == "norm_forward":
        y, mean, rstd = ssd.ssd_layer_norm_forward(s["x"], s["weight"], s["bias"], s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    return ssd.ssd_layer_norm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], want_dbias=c["bias"])


def _kept(s, batch, seqlen):
    """(batch, seqlen, 1): whether a position is within its row's length, and the lengths."""
    if s["lengths"] is None:
        n = torch.full((batch,), seqlen, device="cuda")
    else:
        n = s["lengths"].long()
    return (torch.arange(seqlen, device="cuda") < n[:, None])[..., None], n


def _conv_terms(s):
    x, W = s["x"].float(), s["case"]["width"]
    b, L, ch = x.shape
    keep, n = _kept(s, b, L)
    before = x.new_zeros(b, W - 1, ch) if s["init"] is None else s["init"].float()
    rows = torch.cat([before, torch.where(keep, x, 0.0)], 1)  # row j + W - 1 is token j
    pre = sum(s["weight"][:, k] * rows[:, k:k + L] for k in range(W))
    return rows, pre if s["bias"] is None else pre + s["bias"], keep, n


def _conv_forward(s):
    T, W = s["x"].dtype, s["case"]["width"]
    rows, pre, keep, n = _conv_terms(s)
    y = torch.where(keep, pre * torch.sigmoid(pre) if s["case"]["silu"] else pre, 0.0).to(T)
    last = (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(-1, -1, y.shape[2])
    y = [v.contiguous() for v in y.split(s["pieces"], -1)]
    return {"y": tuple(y), "final": rows.gather(1, last).to(T)}


def _conv_backward(s):
    T, W = s["x"].dtype, s["case"]["width"]
    rows, pre, keep, n = _conv_terms(s)
    b, L, ch = pre.shape
    g = torch.cat([v.float() for v in s["dy"]], -1)
    if s["case"]["silu"]:
        sig = torch.sigmoid(pre)
        g = g * sig * (1 + pre * (1 - sig))
    g = torch.where(keep, g, 0.0)
    wide = torch.nn.functional.pad(g, (0, 0, W - 1, W - 1))  # row j + W - 1 is token j's
    drows = sum(s["weight"][:, k] * wide[:, W - 1 - k:W - 1 - k + L + W - 1] for k in range(W))
    if s["dfinal"] is not None:
        last = (n[:, None] + torch.arange(W - 1, device="cuda"))[..., None].expand(-1, -1, ch)
        drows = drows.scatter_add(1, last, s["dfinal"].float())
    dweight = torch.stack([(g * rows[:, k:k + L]).sum((0, 1)) for k in range(W)], 1)
    return {"dx": drows[:, W - 1:].to(T), "dweight": dweight, "dbias": g.sum((0, 1)) if s["bias"] is not None else None,
            "dinit": drows[:, :W - 1].to(T) if s["init"] is not None else None}


def _conv_step(s):
    x, state, W = s["x"].float(), s["state"], s["case"]["width"]
    at = torch.arange(len(x), device="cuda") if s["slots"] is None else s["slots"].long()
    live = at >= 0
    rows = torch.cat([state[at.clamp(min=0)].float(), x[:, None]], 1)
    pre = sum(s["weight"][:, k] * rows[:, k] for k in range(W))
    pre = pre if s["bias"] is None else pre + s["bias"]
    y = torch.where(live[:, None], pre * torch.sigmoid(pre) if s["case"]["silu"] else pre, 0.0).to(state.dtype)
    if s["slots"] is None:
        state.copy_(rows[:, 1:])
    else:
        state[at[live]] = rows[live, 1:].to(state.dtype)
    return {"y": tuple(v.contiguous() for v in y.split(s["pieces"], -1)), "state": state}


def _scan(a, b):
    """h[t] = a[t] h[t-1] + b[t] along dimension 1 from zero: pairs of steps are one step of a scan half as long."""
    L = b.shape[1]
    if L == 1:
        return b
    pairs = L // 2 * 2
    a0, a1, b0, b1 = a[:, 0:pairs:2], a[:, 1:pairs:2], b[:, 0:pairs:2], b[:, 1:pairs:2]
    odd = _scan(a0 * a1, a1 * b0 + b1)
    h = torch.empty_like(b)
    h[:, 1:pairs:2] = odd
    h[:, 0] = b[:, 0]
    h[:, 2::2] = a[:, 2::2] * odd[:, :(L - 1) // 2] + b[:, 2::2]
    return h


def _effective_dt(s):
    dt = s["dt"].float()
    dt = dt if s["bias"] is None else dt + s["bias"]
    return dt.clamp(min=0) + torch.log1p(torch.exp(-dt.abs())) if s["case"]["softplus"] else dt


def _by_channel(v, channels):
    """(..., groups, dstate) in 32 bits, each group's row given to its channels: (..., channels, dstate)."""
    return v.float().repeat_interleave(channels // v.shape[-2], -2)


def _selective_terms(s):
    x = s["x"].float()
    b, L, ch = x.shape
    keep, _ = _kept(s, b, L)
    dt = torch.where(keep, _effective_dt(s), 0.0)  # a token past the length keeps the state
    x = torch.where(keep, x, 0.0)
    B, C = (torch.where(keep[..., None], _by_channel(s[k], ch), 0.0) for k in "BC")
    a = torch.exp(dt[..., None] * s["A"])
    bx = (dt * x)[..., None] * B
    if s["init"] is not None:
        h = _scan(a, torch.cat([bx[:, :1] + a[:, :1] * s["init"][:, None], bx[:, 1:]], 1))
    else:
        h = _scan(a, bx)
    return x, dt, a, bx, B, C, h, keep


def _selective_forward(s):
    x, _, _, _, _, C, h, keep = _selective_terms(s)
    y = (C * h).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": torch.where(keep, y, 0.0).to(s["x"].dtype), "final": h[:, -1].contiguous()}


def _selective_backward(s):
    x, dt, a, bx, B, C, h, keep = _selective_terms(s)
    T, (b, L, ch, N), G = s["x"].dtype, h.shape, s["case"]["ngroups"]
    g = torch.where(keep, s["dy"].float(), 0.0)
    out = {}
    if s["z"] is not None:
        z = torch.where(keep, s["z"].float(), 0.0)
        sig = torch.sigmoid(z)
        out["dz"] = (g * ((C * h).sum(-1) + s["D"] * x) * sig * (1 + z * (1 - sig))).to(T)
        g = g * z * sig
    mu = g[..., None] * C
    if s["dfinal"] is not None:
        mu = torch.cat([mu[:, :-1], mu[:, -1:] + s["dfinal"][:, None]], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    lam = _scan(after.flip(1), mu.flip(1)).flip(1)  # the gradient of the state after each token
    held = lam * (h - bx)  # times a h of the token before
    by_b = (lam * B).sum(-1)
    ddt = torch.where(keep, (held * s["A"]).sum(-1) + by_b * x, 0.0)
    if s["case"]["softplus"]:
        raw = s["dt"].float() + (0.0 if s["bias"] is None else s["bias"])
        ddt = torch.where(keep, ddt * torch.sigmoid(raw), 0.0)
    out.update(dx=torch.where(keep, by_b * dt + g * s["D"], 0.0).to(T), ddt=ddt.to(T), dA=(held * dt[..., None]).sum((0, 1)),
               dB=torch.where(keep[..., None], (lam * (dt * x)[..., None]).unflatten(2, (G, -1)).sum(3), 0.0),
               dC=(h * g[..., None]).unflatten(2, (G, -1)).sum(3), dD=(g * x).sum((0, 1)),
               ddt_bias=ddt.sum((0, 1)) if s["bias"] is not None else None,
               dinit=a[:, 0] * lam[:, 0] if s["init"] is not None else None)
    return out


def _selective_step(s):
    x, state = s["x"].float(), s["state"]
    ch = x.shape[1]
    at = torch.arange(len(x), device="cuda") if s["slots"] is None else s["slots"].long()
    live = at >= 0
    dt = _effective_dt(s)
    h = torch.exp(dt[..., None] * s["A"]) * state[at.clamp(min=0)] + (dt * x)[..., None] * _by_channel(s["B"], ch)
    y = (_by_channel(s["C"], ch) * h).sum(-1) + s["D"] * x
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    if s["slots"] is None:
        state.copy_(h)
    else:
        state[at[live]] = h[live]
    return {"y": torch.where(live[:, None], y, 0.0).to(s["x"].dtype), "state": state}


def _norm_forward(s):
    x = s["x"].float()
    mean = x.mean(-1)
    off = x - mean[:, None]
    rstd = torch.rsqrt(off.square().mean(-1) + s["eps"])
    y = off * rstd[:, None] * s["weight"]
    return {"y": (y if s["bias"] is None else y + s["bias"]).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_backward(s):
    x, g = s["x"].float(), s["dy"].float()
    xhat = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gw = g * s["weight"]
    dx = s["rstd"][:, None] * (gw - gw.mean(-1, keepdim=True) - xhat * (gw * xhat).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dweight": (g * xhat).sum(0), "dbias": g.sum(0) if s["case"]["bias"] else None}


PLAIN = {"conv_forward": _conv_forward, "conv_backward": _conv_backward, "conv_step": _conv_step,
         "selective_forward": _selective_forward, "selective_backward": _selective_backward, "selective_step": _selective_step,
         "norm_forward": _norm_forward, "norm_backward": _norm_backward}


# ------------------------------------------------------------------------------------------------ what it takes


def work(case):
    """Bytes: every input read once and every output written once.  Operations: a multiply-add is two, an
    exponential (and a sigmoid's or a softplus's) one each."""
    e, op = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]], case["op"]
    if op.startswith("conv"):
        pieces, W = [int(n) for n in case["pieces"].split(",")], case["width"]
        ch = sum(pieces)
        n = case["batch"] * case.get("seqlen", 1) * ch
        edge = case["batch"] * (W - 1) * ch * e
        pre = 2 * W + 4 * case["silu"]
        small = ch * (W + 1) * 4
        if op == "conv_step":
            return {"bytes": 2 * n * e + 2 * edge + small, "flops": n * pre}
        if op == "conv_forward":
            return {"bytes": 2 * n * e + edge * (1 + case["init"]) + small, "flops": n * pre}
        tail = case["batch"] * case["seqlen"] * (ch - pieces[0])
        return {"bytes": 3 * n * e + tail * (4 - e) + 3 * edge * case["init"] + 2 * small, "flops": n * (pre + 4 * W + 6)}
    if op.startswith("selective"):
        rows, ch, G, N = case["batch"] * case.get("seqlen", 1), case["channels"], case["ngroups"], case["dstate"]
        n, bc, state = rows * ch, rows * G * N, case["batch"] * ch * N * 4
        gate = int(case["gate"])
        small = ch * (N + 2) * 4
        if op == "selective_step":
            return {"bytes": n * e * (3 + gate) + 2 * bc * e + 2 * state + small, "flops": n * (7 * N + 8)}
        if op == "selective_forward":
            return {"bytes": n * e * (3 + gate) + 2 * bc * e + state * (1 + case["init"]) + small, "flops": n * (7 * N + 8)}
        return {"bytes": n * e * (5 + 2 * gate) + bc * (2 * e + 8) + 3 * state * case["init"] + 2 * small,
                "flops": n * (22 * N + 20)}
    n = case["rows"] * case["width"]
    if op == "norm_forward":
        return {"bytes": 2 * n * e + 8 * case["rows"] + 8 * case["width"], "flops": 8 * n}
    return {"bytes": 3 * n * e + 8 * case["rows"] + 12 * case["width"], "flops": 14 * n}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op.startswith("conv"):
        if op == "conv_step":
            return _exact_conv_step(case, s)
        s["dy"] = [v.double() for v in s.get("dy", [])]
        return _exact_conv(case, s)
    if op.startswith("selective"):
        if op == "selective_step":
            return _exact_selective_step(case, s)
        return _exact_selective(case, s)
    x = s["x"].clone().requires_grad_()
    w = s["weight"].clone().requires_grad_()
    bias = torch.zeros_like(w) if s["bias"] is None else s["bias"]
    bias = bias.clone().requires_grad_()
    y = torch.nn.functional.layer_norm(x, (case["width"],), w, bias, s["eps"])
    if op == "norm_forward":
        return {"y": y.detach(), "mean": x.mean(-1).detach(), "rstd": (x.var(-1, correction=0) + s["eps"]).rsqrt().detach()}
    dx, dw, db = torch.autograd.grad(y, [x, w, bias], s["dy"])
    return {"dx": dx, "dweight": dw, "dbias": db if case["bias"] else None}


def _exact_conv(case, s):
    W, L, pieces = case["width"], case["seqlen"], s["pieces"]
    with torch.enable_grad():
        x = s["x"].clone().requires_grad_()
        w = s["weight"].clone().requires_grad_()
        ch = w.shape[0]
        bias = (torch.zeros(ch, dtype=torch.float64, device="cuda") if s["bias"] is None else s["bias"]).clone().requires_grad_()
        init = (torch.zeros(case["batch"], W - 1, ch, dtype=torch.float64, device="cuda") if s["init"] is None else s["init"])
        init = init.clone().requires_grad_()
        ys, finals = [], []
        for b in range(case["batch"]):  # one row at its own length
            n = L if s["lengths"] is None else int(s["lengths"][b])
            rows = torch.cat([init[b], x[b, :n]])
            y = torch.nn.functional.conv1d(rows.T[None], w[:, None], bias, groups=ch)[0].T if n else rows[:0]
            if case["silu"]:
                y = torch.nn.functional.silu(y)
            ys.append(torch.nn.functional.pad(y, (0, 0, 0, L - n)))
            finals.append(rows[len(rows) - (W - 1):])
        y, final = torch.stack(ys), torch.stack(finals)
        if case["op"] == "conv_forward":
            return {"y": tuple(v.detach().contiguous() for v in y.split(pieces, -1)), "final": final.detach()}
        dfinal = torch.zeros_like(final) if s["dfinal"] is None else s["dfinal"]
        dx, dw, db, dinit = torch.autograd.grad([y, final], [x, w, bias, init], [torch.cat(s["dy"], -1), dfinal])
    return {"dx": dx, "dweight": dw, "dbias": db if s["bias"] is not None else None, "dinit": dinit if s["init"] is not None else None}


def _exact_conv_step(case, s):
    y = torch.zeros_like(s["x"])
    state = s["state"].clone()
    slots = range(case["batch"]) if s["slots"] is None else s["slots"].tolist()
    for i, at in enumerate(slots):
        if at < 0:
            continue
        taps = torch.cat([s["state"][at], s["x"][i:i + 1]])
        y[i] = (taps * s["weight"].T).sum(0) + (0.0 if s["bias"] is None else s["bias"])
        state[at] = taps[1:]
    y = y / (1 + torch.exp(-y)) if case["silu"] else y
    live = torch.tensor([at >= 0 for at in slots], device="cuda")
    return {"y": tuple(v.contiguous() for v in (y * live[:, None]).split(s["pieces"], -1)), "state": state}


def _exact_token(s, case, leaf, x, dt, B, C, h, z):
    """The state after one token, and its output."""
    ch = x.shape[-1]
    dt = dt if leaf["bias"] is None else dt + leaf["bias"]
    dt = torch.nn.functional.softplus(dt) if case["softplus"] else dt
    per = ch // case["ngroups"]
    B, C = (v.unsqueeze(2).expand(-1, -1, per, -1).reshape(len(x), ch, -1) for v in (B, C))
    h = torch.addcmul((dt * x).unsqueeze(-1) * B, torch.exp(dt.unsqueeze(-1) * leaf["A"]), h)
    y = torch.einsum("bcn,bcn->bc", C, h) + leaf["D"] * x
    return h, y if z is None else y * torch.nn.functional.silu(z)


def _exact_selective_step(case, s):
    slots = torch.arange(case["batch"], device="cuda") if s["slots"] is None else s["slots"].long()
    rows = (slots >= 0).nonzero()[:, 0]
    at = slots[rows]
    h, out = _exact_token(s, case, s, s["x"][rows], s["dt"][rows], s["B"][rows], s["C"][rows], s["state"][at],
                          None if s["z"] is None else s["z"][rows])
    y, state = torch.zeros_like(s["x"]), s["state"].clone()
    y[rows], state[at] = out, h
    return {"y": y, "state": state}


def _exact_selective(case, s):
    """Token by token; the gradients by differentiating that."""
    grad = case["op"] == "selective_backward"
    elements = case["batch"] * case["channels"] * case["dstate"]
    if case["seqlen"] * (elements * 4e-10 + 2.5e-4) * (4 if grad else 1) > 20 or grad and case["seqlen"] * elements * 8 * 8 > 6e10:
        return None
    names = ("x", "dt", "A", "B", "C", "D", "bias", "z", "init")
    leaf = {k: None if s[k] is None else s[k].clone().requires_grad_(grad) for k in names}
    b, L = case["batch"], case["seqlen"]
    with torch.set_grad_enabled(grad):
        h = leaf["init"] if leaf["init"] is not None else s["x"].new_zeros(b, case["channels"], case["dstate"])
        ys = []
        tok = {k: [None] * L if leaf[k] is None else leaf[k].unbind(1) for k in ("x", "dt", "B", "C", "z")}
        for t in range(L):
            new, y = _exact_token(s, case, leaf, tok["x"][t], tok["dt"][t], tok["B"][t], tok["C"][t], h, tok["z"][t])
            if s["lengths"] is not None:
                live = (t < s["lengths"])[:, None]
                new, y = torch.where(live[..., None], new, h), torch.where(live, y, 0.0)
            h = new
            ys.append(y)
        y = torch.stack(ys, 1)
        if not grad:
            return {"y": y, "final": h}
        wanted = [k for k in names if leaf[k] is not None]
        outs, given = ([y, h], [s["dy"], s["dfinal"]]) if s["dfinal"] is not None else ([y], [s["dy"]])
        got = dict(zip(wanted, torch.autograd.grad(outs, [leaf[k] for k in wanted], given)))
    out = {"dx": got["x"], "ddt": got["dt"], "dA": got["A"], "dB": got["B"], "dC": got["C"], "dD": got["D"],
           "ddt_bias": got.get("bias"), "dinit": got.get("init")}
    if "z" in got:
        out["dz"] = got["z"]
    return out
