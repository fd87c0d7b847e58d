"""The cases that the gated recurrence, the grouped norm and the rotary positions are measured on, with their plain forms.

  gated_*   the gated linear recurrence, one state per channel: h <- a h + sqrt(1 - a^2) sigmoid(i) x with
            a = exp(A sigmoid(r)); prompts or training rows, its gradient, single tokens;
  group_*   the norm over groups of a token's channels (group norm, channels last) with its activation: a gate
            silu(z) in front of the norm or behind it, or silu of the output; its gradient;
  rotary_*  rotary positions on a scan's B and C (or queries and keys): interleaved and half layouts, part of the
            head, scaled for long contexts; the gradient; single tokens.

`run` makes the library's calls where `own` is true, and computes the same from elementary torch operations in
32 bits (angles in 64), rounded once at the end, where it is false.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SPAN = 64  # tokens between the states that the recurrence's forward pass keeps for its gradient


def listed():
    return [
        # a short prompt of a small layer in 32 bits, its state carried in (latency counts)
        dict(name="gated_prompt_short", op="gated_forward", dtype="f32", batch=1, seqlen=512, channels=256, offset=0, init=True,
             ragged=False, states=False),
        # a layer's training forward, with the states that its gradient starts from; the gates are slices of a projection's rows
        dict(name="gated_prompt", op="gated_forward", dtype="bf16", batch=2, seqlen=4096, channels=4096, offset=4096, init=False,
             ragged=False, states=True),
        # prompts of unlike lengths padded to one row length, one of them empty; odd sizes
        dict(name="gated_ragged", op="gated_forward", dtype="f16", batch=5, seqlen=1777, channels=1530, offset=3, init=True,
             ragged=True, states=False),
        # one long document
        dict(name="gated_long", op="gated_forward", dtype="bf16", batch=1, seqlen=65536, channels=2048, offset=2048, init=True,
             ragged=False, states=False),
        # the gradient of a training step
        dict(name="gated_grad", op="gated_backward", dtype="bf16", batch=2, seqlen=4096, channels=4096, offset=4096, init=False,
             ragged=False, states=True),
        # one token of 256 sequences, their states in slots of a pool, a few rows of the batch idle
        dict(name="gated_decode", op="gated_step", dtype="bf16", batch=256, channels=4096, offset=4096, slots=True),
        # the norm behind a scan: 64 heads of 64 in 8 groups, gated by z in front of the norm, no mean; z is a slice of the
        # input projection's rows
        dict(name="group_prompt", op="group_forward", dtype="bf16", rows=8192, width=4096, groups=8, gate="before", rms=True,
             bias=False, tail=256),
        # the gradient at the same layer
        dict(name="group_grad", op="group_backward", dtype="bf16", rows=8192, width=4096, groups=8, gate="before", rms=True, bias=False,
             tail=256),
        # a norm per head with mean, bias and silu of its output, of widths that fit no vector
        dict(name="group_heads", op="group_forward", dtype="f16", rows=3554, width=1530, groups=15, gate="silu", rms=False, bias=True,
             tail=3),
        # B and C of one very long document, 8 groups of 256, turned at positions scaled for the length
        dict(name="rotary_long", op="rotary_forward", dtype="bf16", batch=1, seqlen=262144, groups=8, groups2=8, dstate=256, turned=256,
             interleaved=False, positions="start", factor=8.0, tail=128, ragged=False),
        # the gradients of B and C as the scan's backward pass returns them, in 32 bits
        dict(name="rotary_grad", op="rotary_backward", dtype="f32", batch=2, seqlen=4096, groups=1, groups2=1, dstate=128, turned=64,
             interleaved=True, positions="none", factor=1.0, tail=0, ragged=False),
        # one token of 256 sequences at positions of their own
        dict(name="rotary_decode", op="rotary_step", dtype="bf16", batch=256, groups=8, groups2=8, dstate=128, turned=128, interleaved=False,
             positions="start", factor=1.0, tail=64),
    ]


def _size(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm; half of them are a multiple of 8."""
    n = max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))
    return max(lo, min(hi, (n + 4) // 8 * 8)) if n > 16 and rng.random() < 0.5 else n


def draw(rng):
    cap = max(work(c)["bytes"] for c in listed()) / 4
    while True:
        case = _draw(rng)
        if work(case)["bytes"] <= cap:
            return case


def _draw(rng):
    op = rng.choice(["gated_forward", "gated_forward", "gated_backward", "gated_backward", "gated_step", "group_forward",
                     "group_backward", "rotary_forward", "rotary_backward", "rotary_step"])
    case = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    coin = lambda: rng.random() < 0.5  # noqa: E731
    if op.startswith("gated"):
        ch = _size(rng, 64, 8192)
        case.update(channels=ch, offset=rng.choice([0, ch, 3]))
        if op == "gated_step":
            case.update(batch=_size(rng, 1, 512), slots=coin())
        else:
            case.update(batch=rng.choice([1, 2, 3, 8]), seqlen=_size(rng, 1, 65536 if op == "gated_forward" else 16384), init=coin(),
                        ragged=coin(), states=coin())
    elif op.startswith("group"):
        groups = rng.choice([1, 1, 2, 3, 8, 15, 64])
        case.update(rows=_size(rng, 1, 65536), groups=groups, width=groups * _size(rng, max(8, 64 // groups), 16384 // groups),
                    gate=rng.choice(["none", "silu", "after", "before", "before"]), rms=coin(), bias=coin(), tail=rng.choice([0, 0, 64, 3]))
    else:
        n = 2 * _size(rng, 16, 128)
        case.update(groups=rng.choice([1, 2, 8, 32]), groups2=rng.choice([1, 2, 8]), dstate=n, turned=rng.choice([n, n, 2 * max(1, n // 4)]),
                    interleaved=coin(), positions=rng.choice(["none", "start", "each"]), factor=rng.choice([1.0, 1.0, 8.0]),
                    tail=rng.choice([0, 0, 64, 3]))
        if op == "rotary_step":
            case.update(batch=_size(rng, 1, 512), positions="start")
        else:
            case.update(batch=rng.choice([1, 2, 3, 8]), seqlen=_size(rng, 1, 131072), ragged=coin())
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


def _frequencies(case):
    """Radians a position, per pair: 10000^(-k / pairs), all of them divided by the factor."""
    pairs = case["turned"] // 2
    return [10000.0 ** (-k / pairs) / case["factor"] for k in range(pairs)]


def prepare(case, seed):
    rand = torch.Generator(device="cuda")
    rand.manual_seed(seed)
    T, op = TYPES[case["dtype"]], case["op"]

    def normal(*shape, dtype=T, scale=1.0):
        return (torch.randn(shape, generator=rand, device="cuda") * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=rand, device="cuda") * (hi - lo) + lo

    s = {"case": case}
    if op.startswith("gated"):
        ch, off = case["channels"], case["offset"]
        rows = (case["batch"],) if op == "gated_step" else (case["batch"], case["seqlen"])
        gates = normal(*rows, off + 2 * ch)
        # at an open gate a channel keeps 0.9 to 0.999 of its state a token
        s.update(x=normal(*rows, ch), r=gates[..., off:off + ch], i=gates[..., off + ch:],
                 A=-torch.exp(uniform(ch, lo=math.log(0.008), hi=math.log(0.84))))
        if op == "gated_step":
            pool, s["slots"] = _slots(case, rand)
            s["state"] = normal(pool, ch, dtype=torch.float32, scale=0.5)
        else:
            s.update(init=normal(case["batch"], ch, dtype=torch.float32, scale=0.5) if case["init"] else None, lengths=_lengths(case, rand))
        if op == "gated_backward":
            s.update(dy=normal(*rows, ch), dfinal=normal(case["batch"], ch, dtype=torch.float32) if case["init"] else None)
            if case["states"]:  # what the forward pass keeps: the state in front of every SPAN tokens
                h = _gated_terms(s, torch.float64)[-2]
                before = torch.zeros_like(h[:, 0]) if s["init"] is None else s["init"].double()
                s["kept"] = torch.cat([before[:, None], h[:, SPAN - 1:case["seqlen"] - 1:SPAN]], 1).float()
            else:
                s["kept"] = None
    elif op.startswith("group"):
        n, w, G = case["rows"], case["width"], case["groups"]
        # a scan's output: channels of unlike scale
        x = normal(n, w + case["tail"], dtype=torch.float32) * torch.exp(normal(w + case["tail"], dtype=torch.float32, scale=0.5))
        s.update(x=(x + normal(n, 1, dtype=torch.float32, scale=0.3)).to(T)[:, :w], weight=1 + normal(w, dtype=torch.float32, scale=0.1),
                 bias=normal(w, dtype=torch.float32, scale=0.1) if case["bias"] else None, eps=1e-5,
                 z=normal(n, w + case["tail"])[:, case["tail"]:] if case["gate"] in ("before", "after") else None)
        if op == "group_backward":
            q = s["x"].double()
            if case["gate"] == "before":
                q = q * s["z"].double() * torch.sigmoid(s["z"].double())
            q = q.unflatten(-1, (G, -1))
            mean = q.mean(-1)
            s["mean"] = None if case["rms"] else mean.float()
            off = q if case["rms"] else q - mean[..., None]
            s["rstd"] = torch.rsqrt(off.square().mean(-1) + s["eps"]).float()
            s["dy"] = normal(n, w)
    else:
        rows = (case["batch"],) if op == "rotary_step" else (case["batch"], case["seqlen"])
        G1, G2, N, tail = case["groups"], case["groups2"], case["dstate"], case["tail"]
        # slices of one projection's rows
        wide = normal(*rows, tail + (G1 + G2) * N)
        s.update(B=wide[..., tail:tail + G1 * N].unflatten(-1, (G1, N)), C=wide[..., tail + G1 * N:].unflatten(-1, (G2, N)))
        if case["positions"] == "none":
            s["positions"] = None
        elif case["positions"] == "start":  # a row's (or a token's) place in a document of up to a million tokens
            s["positions"] = (uniform(case["batch"]) * 1e6).to(torch.int32)
        else:  # documents packed into the rows, each from position 0
            at = torch.arange(case["seqlen"], device="cuda") + (uniform(case["batch"], 1) * 1000).long()
            s["positions"] = (at % 1000).to(torch.int32)
        f = _frequencies(case)
        # the part of a turn that a position adds, in units of 2^-64
        turns = [round(v / (2 * math.pi) * 2.0 ** 64) % 2 ** 64 for v in f]
        s.update(table=torch.tensor([t - 2 ** 64 if t >= 2 ** 63 else t for t in turns], dtype=torch.int64, device="cuda"),
                 frequencies=torch.tensor(f, dtype=torch.float64, device="cuda"), scale=1.0 + 0.1 * math.log(case["factor"]))
        if op != "rotary_step":
            s["lengths"] = _lengths(case, rand)
    return s


# ------------------------------------------------------------------------------------------------ the passes


def run(s):
    return _library(s) if own else PLAIN[s["case"]["op"]](s)


def _library(s):
    import state_space_sequence_ssd_gb300 as ssd
    c, op = s["case"], s["case"]["op"]
    if op == "gated_forward":
        y, final, states = ssd.ssd_gated_forward(s["x"], s["r"], s["i"], s["A"], s["init"], s["lengths"], want_states=c["states"])
        return {"y": y, "final": final, "states": states}
    if op == "gated_backward":
        return ssd.ssd_gated_backward(s["x"], s["r"], s["i"], s["A"], s["dy"], s["init"], s["lengths"], states=s["kept"],
                                      dfinal=s["dfinal"], want_dinit=c["init"])
    if op == "gated_step":
        y = ssd.ssd_gated_step(s["x"], s["r"], s["i"], s["A"], s["state"], s["slots"])
        return {"y": y, "state": s["state"]}
    if op == "group_forward":
        y, mean, rstd = ssd.ssd_group_norm_forward(s["x"], c["groups"], s["weight"], s["bias"], z=s["z"], gate_first=c["gate"] == "before",
                                                   silu=c["gate"] == "silu", rms=c["rms"], eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "group_backward":
        return ssd.ssd_group_norm_backward(s["x"], c["groups"], s["weight"], s["bias"], s["mean"], s["rstd"], s["dy"], z=s["z"],
                                           gate_first=c["gate"] == "before", silu=c["gate"] == "silu")
    if op == "rotary_step":
        return ssd.ssd_rotary_step(s["B"], s["C"], s["table"], s["positions"], interleaved=c["interleaved"], scale=s["scale"])
    call = ssd.ssd_rotary_forward if op == "rotary_forward" else ssd.ssd_rotary_backward
    return call(s["B"], s["C"], s["table"], s["positions"], s["lengths"], interleaved=c["interleaved"], scale=s["scale"])


def _kept(s, batch, seqlen):
    """(batch, seqlen, 1): whether a position is within its row's length."""
    if s["lengths"] is None:
        return torch.ones(batch, seqlen, 1, dtype=torch.bool, device="cuda")
    return (torch.arange(seqlen, device="cuda") < s["lengths"].long()[:, None])[..., None]


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


def _gated_terms(s, to=torch.float32):
    """x, sigmoid(r), sigmoid(i), log a, a, sqrt(1 - a^2), h, and which tokens count; the others keep the state."""
    b, L, _ = s["x"].shape
    keep = _kept(s, b, L)
    x = torch.where(keep, s["x"].to(to), 0.0)
    v, g = torch.sigmoid(s["r"].to(to)), torch.sigmoid(s["i"].to(to))
    u = torch.where(keep, s["A"].to(to) * v, 0.0)
    a, w = torch.exp(u), torch.sqrt(-torch.expm1(2 * u))
    bx = w * g * x
    if s["init"] is not None:
        h = _scan(a, torch.cat([bx[:, :1] + a[:, :1] * s["init"][:, None].to(to), bx[:, 1:]], 1))
    else:
        h = _scan(a, bx)
    return x, v, g, u, a, w, h, keep


def _gated_forward(s):
    *_, h, keep = _gated_terms(s)
    states = None
    if s["case"]["states"]:
        before = torch.zeros_like(h[:, 0]) if s["init"] is None else s["init"]
        states = torch.cat([before[:, None], h[:, SPAN - 1:h.shape[1] - 1:SPAN]], 1)
    return {"y": torch.where(keep, h, 0.0).to(s["x"].dtype), "final": h[:, -1].contiguous(), "states": states}


def _gated_backward(s):
    x, v, g, u, a, w, h, keep = _gated_terms(s)
    T = s["x"].dtype
    mu = torch.where(keep, s["dy"].float(), 0.0)
    if s["dfinal"] is not None:
        mu = torch.cat([mu[:, :-1], mu[:, -1:] + s["dfinal"][:, None]], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    lam = _scan(after.flip(1), mu.flip(1)).flip(1)  # the gradient of the state after each token
    before = torch.zeros_like(h[:, :1]) if s["init"] is None else s["init"][:, None]
    held = torch.where(keep, lam * (u * a * torch.cat([before, h[:, :-1]], 1) - torch.where(w > 0, u * a * a / w, 0.0) * g * x), 0.0)
    return {"dx": torch.where(keep, lam * w * g, 0.0).to(T), "dr": (held * (1 - v)).to(T),
            "di": torch.where(keep, lam * w * x * g * (1 - g), 0.0).to(T), "dA": held.sum((0, 1)) / s["A"],
            "dinit": a[:, 0] * lam[:, 0] if s["init"] is not None else None}


def _gated_step(s):
    state = s["state"]
    at = torch.arange(len(s["x"]), device="cuda") if s["slots"] is None else s["slots"].long()
    live = at >= 0
    u = s["A"] * torch.sigmoid(s["r"].float())
    h = torch.exp(u) * state[at.clamp(min=0)] + torch.sqrt(-torch.expm1(2 * u)) * torch.sigmoid(s["i"].float()) * s["x"].float()
    if s["slots"] is None:
        state.copy_(h)
    else:
        state[at[live]] = h[live]
    return {"y": torch.where(live[:, None], h, 0.0).to(s["x"].dtype), "state": state}


def _group_terms(s):
    """What is normalised, in groups."""
    q = s["x"].float()
    if s["case"]["gate"] == "before":
        z = s["z"].float()
        q = q * z * torch.sigmoid(z)
    return q.unflatten(-1, (s["case"]["groups"], -1))


def _group_forward(s):
    c, q = s["case"], _group_terms(s)
    mean = None
    if not c["rms"]:
        mean = q.mean(-1)
        q = q - mean[..., None]
    rstd = torch.rsqrt(q.square().mean(-1) + s["eps"])
    y = (q * rstd[..., None]).flatten(-2) * s["weight"]
    y = y if s["bias"] is None else y + s["bias"]
    if c["gate"] == "silu":
        y = y * torch.sigmoid(y)
    if c["gate"] == "after":
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _group_backward(s):
    c, q, T = s["case"], _group_terms(s), s["x"].dtype
    rstd = s["rstd"][..., None]
    xhat = ((q if c["rms"] else q - s["mean"][..., None]) * rstd).flatten(-2)
    g, out = s["dy"].float(), {}
    pre = xhat * s["weight"] if s["bias"] is None else xhat * s["weight"] + s["bias"]
    if c["gate"] == "silu":
        sig = torch.sigmoid(pre)
        g = g * sig * (1 + pre * (1 - sig))
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        slope = sig * (1 + z * (1 - sig))
    if c["gate"] == "after":
        out["dz"] = (g * pre * slope).to(T)
        g = g * z * sig
    gw, xh = (g * s["weight"]).unflatten(-1, (c["groups"], -1)), xhat.unflatten(-1, (c["groups"], -1))
    dq = gw - xh * (gw * xh).mean(-1, keepdim=True)
    dq = ((dq if c["rms"] else dq - gw.mean(-1, keepdim=True)) * rstd).flatten(-2)
    if c["gate"] == "before":
        out["dz"] = (dq * s["x"].float() * slope).to(T)
        dq = dq * z * sig
    out.update(dx=dq.to(T), dweight=(g * xhat).sum(0), dbias=g.sum(0) if s["bias"] is not None else None)
    return out


def _turned(t, cos, sin, case):
    """The first `turned` entries of each head as pairs, turned; the others as they are.  cos, sin (..., 1, pairs)."""
    t = t.float()
    rot, rest = t[..., :case["turned"]], t[..., case["turned"]:]
    if case["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = rot.chunk(2, -1)
        rot = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([rot, rest], -1)


def _rotary(s):
    c, B = s["case"], s["B"]
    p = s["positions"]
    if c["op"] == "rotary_step":
        at, keep = p.double(), None
    else:
        at = torch.arange(B.shape[1], device="cuda", dtype=torch.float64).expand(B.shape[:2])
        if p is not None:
            at = p.double() if p.dim() == 2 else at + p.double()[:, None]
        keep = _kept(s, *B.shape[:2])[..., None]
    angle = at[..., None, None] * s["frequencies"]
    cos, sin = (s["scale"] * torch.cos(angle)).float(), (s["scale"] * torch.sin(angle)).float()
    if c["op"] == "rotary_backward":
        sin = -sin
    out = [_turned(t, cos, sin, c) for t in (B, s["C"])]
    return tuple((t if keep is None else torch.where(keep, t, 0.0)).to(B.dtype) for t in out)


PLAIN = {"gated_forward": _gated_forward, "gated_backward": _gated_backward, "gated_step": _gated_step, "group_forward": _group_forward,
         "group_backward": _group_backward, "rotary_forward": _rotary, "rotary_backward": _rotary, "rotary_step": _rotary}


# ------------------------------------------------------------------------------------------------ what it takes


def work(case):
    """Bytes: every input read once and every output written once.  Operations: a multiply-add is two, an
    exponential, a root or a quotient one each."""
    e, op = {"bf16": 2, "f16": 2, "f32": 4}[case["dtype"]], case["op"]
    if op.startswith("gated"):
        b, L, ch = case["batch"], case.get("seqlen", 1), case["channels"]
        n, state = b * L * ch, 4 * b * ch
        if op == "gated_step":
            return {"bytes": 4 * n * e + 2 * state + 4 * ch, "flops": 16 * n}
        kept = case["states"] * state * -(-L // SPAN)
        if op == "gated_forward":
            return {"bytes": 4 * n * e + (1 + case["init"]) * state + kept + 4 * ch, "flops": 16 * n}
        return {"bytes": 7 * n * e + (3 if case["init"] else 0) * state + kept + 8 * ch, "flops": 38 * n}
    if op.startswith("group"):
        n, stats = case["rows"] * case["width"], 4 * case["rows"] * case["groups"] * (1 if case["rms"] else 2)
        gated = case["gate"] in ("before", "after")
        weights = 4 * case["width"] * (1 + case["bias"])
        if op == "group_forward":
            return {"bytes": (2 + gated) * n * e + stats + weights, "flops": (8 + 5 * (case["gate"] != "none")) * n}
        return {"bytes": (3 + 2 * gated) * n * e + stats + 2 * weights, "flops": (14 + 10 * (case["gate"] != "none")) * n}
    rows = case["batch"] * case.get("seqlen", 1)
    n = rows * (case["groups"] + case["groups2"]) * case["dstate"]
    places = {"none": 0, "start": 4 * case["batch"], "each": 4 * rows}[case["positions"]]
    return {"bytes": 2 * n * e + places + 4 * case["turned"], "flops": 3 * n + 4 * rows * case["turned"]}


# ------------------------------------------------------------------------------------------------ in 64 bits


def exact(case, seed):
    s = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in prepare(case, seed).items()}
    op = case["op"]
    if op == "gated_step":
        return _exact_gated_step(case, s)
    if op.startswith("gated"):
        return _exact_gated(case, s)
    if op.startswith("group"):
        return _exact_group(case, s)
    return _exact_rotary(case, s)


def _exact_token(leaf):
    """Decay and input of every token."""
    decay = leaf["A"] / (1 + torch.exp(-leaf["r"]))
    return torch.exp(decay), (1 - torch.exp(2 * decay)).sqrt() * leaf["x"] / (1 + torch.exp(-leaf["i"]))


def _exact_gated_step(case, s):
    slots = torch.arange(case["batch"], device="cuda") if s["slots"] is None else s["slots"].long()
    rows = (slots >= 0).nonzero()[:, 0]
    a, b = _exact_token({"A": s["A"], **{k: s[k][rows] for k in ("x", "r", "i")}})
    y, state = torch.zeros_like(s["x"]), s["state"].clone()
    y[rows] = state[slots[rows]] = a * s["state"][slots[rows]] + b
    return {"y": y, "state": state}


def _exact_gated(case, s):
    """Token by token; the gradients by differentiating that."""
    grad, b, L, ch = case["op"] == "gated_backward", case["batch"], case["seqlen"], case["channels"]
    if L * (b * ch * 1e-10 + 3e-5) * (8 if grad else 1) > 20 or b * L * ch * 8 * (16 if grad else 6) > 8e10:
        return None
    leaf = {k: None if s[k] is None else s[k].clone().requires_grad_(grad) for k in ("x", "r", "i", "A", "init")}
    with torch.set_grad_enabled(grad):
        h = s["x"].new_zeros(b, ch) if leaf["init"] is None else leaf["init"]
        decay, bx = (v.unbind(1) for v in _exact_token(leaf))
        ys, states = [], []
        for t in range(L):
            if t % SPAN == 0:
                states.append(h.detach())
            new = torch.addcmul(bx[t], decay[t], h)
            if s["lengths"] is None:
                h = new
                ys.append(h)
            else:
                live = (t < s["lengths"])[:, None]
                h = torch.where(live, new, h)
                ys.append(torch.where(live, new, 0.0))
        y = torch.stack(ys, 1)
        if not grad:
            return {"y": y, "final": h, "states": torch.stack(states, 1) if case["states"] else None}
        wanted = [k for k in leaf if leaf[k] is not None]
        outs, given = ([y, h], [s["dy"], s["dfinal"]]) if s["dfinal"] is not None else ([y], [s["dy"]])
        got = dict(zip(wanted, torch.autograd.grad(outs, [leaf[k] for k in wanted], given)))
    return {"dx": got["x"], "dr": got["r"], "di": got["i"], "dA": got["A"], "dinit": got.get("init")}


def _exact_group(case, s):
    grad = case["op"] == "group_backward"
    leaf = {k: None if s[k] is None else s[k].clone().requires_grad_(grad) for k in ("x", "z", "weight", "bias")}
    with torch.set_grad_enabled(grad):
        q = leaf["x"]
        if case["gate"] == "before":
            q = q * torch.nn.functional.silu(leaf["z"])
        q = q.reshape(case["rows"], case["groups"], -1)
        mean = q.mean(-1)
        square = (q ** 2).mean(-1) if case["rms"] else q.var(-1, correction=0)
        rstd = 1 / (square + s["eps"]).sqrt()
        y = ((q if case["rms"] else q - mean[..., None]) * rstd[..., None]).reshape(s["x"].shape) * leaf["weight"]
        y = y if leaf["bias"] is None else y + leaf["bias"]
        if case["gate"] == "silu":
            y = torch.nn.functional.silu(y)
        if case["gate"] == "after":
            y = y * torch.nn.functional.silu(leaf["z"])
        if not grad:
            return {"y": y, "mean": None if case["rms"] else mean, "rstd": rstd}
        wanted = [k for k in leaf if leaf[k] is not None]
        got = dict(zip(wanted, torch.autograd.grad(y, [leaf[k] for k in wanted], s["dy"])))
    out = {"dx": got["x"], "dweight": got["weight"], "dbias": got.get("bias")}
    if "z" in got:
        out["dz"] = got["z"]
    return out


def _exact_rotary(case, s):
    if s["B"].numel() + s["C"].numel() > 2 ** 30:
        return None
    step = case["op"] == "rotary_step"
    B, C = (t[:, None] if step else t for t in (s["B"], s["C"]))
    b, L = B.shape[:2]
    at = torch.zeros(b, L, dtype=torch.int64, device="cuda") if step else torch.arange(L, device="cuda").repeat(b, 1)
    if s["positions"] is not None:
        p = s["positions"].long()
        at = p if p.dim() == 2 else at + p[:, None]
    turn = torch.polar(torch.full((), s["scale"], dtype=torch.float64, device="cuda"), at[..., None] * s["frequencies"])
    turn = turn.conj() if case["op"] == "rotary_backward" else turn
    if not step and s["lengths"] is not None:
        live = at.new_tensor(range(L))[None, :, None] < s["lengths"].long()[:, None, None]
    out = []
    for t in (B, C):
        y, n = t.clone(), case["turned"]
        first = slice(0, n, 2) if case["interleaved"] else slice(0, n // 2)
        second = slice(1, n, 2) if case["interleaved"] else slice(n // 2, n)
        pair = torch.complex(t[..., first].contiguous(), t[..., second].contiguous()) * turn[:, :, None]
        y[..., first], y[..., second] = pair.real, pair.imag
        if not step and s["lengths"] is not None:
            y = torch.where(live[..., None], y, 0.0)
        out.append(y[:, 0] if step else y)
    return tuple(out)
