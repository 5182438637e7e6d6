"""The measured cases of two further sequence operators and their plain forms.

Group norm with an activation over positions in channels-last order, and a
gated linear recurrence along the positions, each with its gradients: a
recurrent block of a sequence or image model, next to a deformable
convolution.  Sizes follow the package's own workloads (the layer's
16 x 512 with 83 output positions, the long sequence 8 x 256 x 16384, the
depthwise 16 x 512 x 4092, the strided layer's 32 x 1024 x 1024 output,
64 x 64 and 28 x 28 images).

With ``own`` false, ``run`` computes an operator in its plain form: elementary
torch operations in 32 bits, rounded once at the end.  With ``own`` true it
calls the package's operators on the same state.
"""
import math

import torch

own = False

_TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_EPS = 1e-5
_EVERY = 64  # the recurrence keeps its state ahead of every 64th position for the backward pass


# ---- cases -------------------------------------------------------------------

def _gn(op, B, S, C, groups, dtype, activation="", ragged=False):
    """S = 0: rows [B, C]; else [B, S, C].  ragged: statistics over the first positions of each sequence only."""
    return {"op": op, "B": B, "S": S, "C": C, "groups": groups, "dtype": dtype, "activation": activation, "ragged": ragged}


def _rec(op, B, L, C, dtype, blend=False, reverse=False, ragged=False):
    return {"op": op, "B": B, "L": L, "C": C, "dtype": dtype, "blend": blend, "reverse": reverse, "ragged": ragged}


def listed():
    return [
        # one new position of each of 16 sequences, 8 heads normalised one by one after the recurrence: latency
        dict(_gn("gn_fwd", 16, 0, 512, 8, "f32", "silu"), name="gn_fwd_step"),
        # 64 x 64 images between two convolutions
        dict(_gn("gn_fwd", 8, 4096, 512, 32, "bf16", "silu"), name="gn_fwd_image"),
        # the long sequence in full precision, one norm over all of its channels and positions
        dict(_gn("gn_fwd", 8, 16384, 256, 1, "f32"), name="gn_fwd_long"),
        # padded batches of the depthwise layer's positions, an odd number of channels in groups of 15
        dict(_gn("gn_fwd", 13, 4092, 255, 17, "bf16", "relu", ragged=True), name="gn_fwd_odd"),
        # training on 28 x 28 images
        dict(_gn("gn_bwd", 32, 784, 512, 32, "f32", "silu"), name="gn_bwd_image"),
        # training on the strided layer's output taken as 32 x 1024 tokens, 16 heads normalised one by one
        dict(_gn("gn_bwd", 32768, 0, 1024, 16, "bf16"), name="gn_bwd_tokens"),
        # one new position of each of 16 sequences from their states: latency
        dict(_rec("rec_fwd", 16, 1, 512, "f32"), name="rec_step"),
        # the long bf16 sequences
        dict(_rec("rec_fwd", 8, 16384, 256, "bf16", blend=True), name="rec_fwd_long"),
        # the strided layer's output, read from its end
        dict(_rec("rec_fwd", 32, 1024, 1024, "f32", reverse=True), name="rec_fwd_tokens"),
        # training on the layer's 83 output positions in full precision
        dict(_rec("rec_bwd", 16, 83, 512, "f32", blend=True), name="rec_bwd_layer"),
        # training on the long bf16 sequences
        dict(_rec("rec_bwd", 8, 16384, 256, "bf16"), name="rec_bwd_long"),
        # training on padded batches of the depthwise layer's positions, an odd number of channels, read from their ends
        dict(_rec("rec_bwd", 13, 4092, 511, "f32", blend=True, reverse=True, ragged=True), name="rec_bwd_odd"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gn_fwd", "gn_bwd", "rec_fwd", "rec_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("gn_fwd", "gn_bwd"):
        groups = rng.choice([1, 4, 8, 16, 17, 32])
        C = groups * _log(rng, max(1, 32 // groups), 2048 // groups)
        S = 0 if rng.random() < 0.2 else _log(rng, 2, 16384)
        room = max(1, (1 << 25) // (C * max(1, S)))
        B = _log(rng, 1, min(32768, room) if S == 0 else min(64, room))
        # the gradient of relu jumps at 0, where roundings alone decide: it is no case to compare values of
        act = rng.choice(["", "silu"] if op == "gn_bwd" else ["", "relu", "silu"])
        return _gn(op, B, S, C, groups, dtype, act, S > 0 and rng.random() < 0.3)
    C, L = _log(rng, 16, 2048), _log(rng, 1, 16384)
    B = _log(rng, 1, max(1, min(64, (1 << 25) // (C * L))))
    return _rec(op, B, L, C, dtype, rng.random() < 0.5, rng.random() < 0.5, L > 1 and rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------

def _lengths(B, n):
    """The ragged lengths: evenly spread from a quarter of n up to n."""
    lo = max(1, n // 4)
    return [lo + (n - lo) * (b + 1) // B for b in range(B)]


def _lens(case, n, gen):
    """The ragged lengths, dealt out by the seed."""
    if not case["ragged"]:
        return None
    order = torch.randperm(case["B"], generator=gen, device=gen.device)
    return torch.tensor(_lengths(case["B"], n), dtype=torch.int32, device=gen.device)[order].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)

    op, B, C = case["op"], case["B"], case["C"]
    s = dict(case)
    if op in ("gn_fwd", "gn_bwd"):
        shape = (B, case["S"], C) if case["S"] else (B, C)
        s["x"] = (randn(*shape) * 1.5 + 0.25).to(dt)
        s["weight"] = (1 + 0.2 * randn(C)).to(dt)
        s["bias"] = (0.2 * randn(C)).to(dt)
        s["lens"] = _lens(case, case["S"], gen)
        if op == "gn_bwd":
            s["g"] = randn(*shape).to(dt)
            x, see, n = _grouped(s, s["x"].float())
            s["mean"], s["rstd"] = _statistics(x, see, n)
        return s
    L = case["L"]
    s["x"] = randn(B, L, C).to(dt)
    # forget gates whose channels remember from a few positions to some hundred
    s["gate"] = (randn(B, L, C) + torch.linspace(0.0, 5.0, C, device="cuda")).to(dt)
    s["state"] = randn(B, C)
    s["lens"] = _lens(case, L, gen)
    if op == "rec_bwd":
        s["g"] = randn(B, L, C).to(dt)
        s["g_last"] = randn(B, C)
        s["states"] = _plain_recurrence(s)["states"]
    return s


# ---- plain forms -------------------------------------------------------------

def _grouped(s, x):
    """x as [B, S, groups, C / groups], which positions count ([B, S, 1, 1], or None: all) and how many elements of a group do."""
    B, C, G = s["B"], s["C"], s["groups"]
    x = x.view(B, max(1, s["S"]), G, C // G)
    if s["lens"] is None:
        return x, None, x.shape[1] * x.shape[3]
    see = torch.arange(x.shape[1], device="cuda").view(1, -1, 1, 1) < s["lens"].view(-1, 1, 1, 1)
    return x, see, (s["lens"] * x.shape[3]).float().view(-1, 1)


def _kept(t, see):
    return t if see is None else torch.where(see, t, torch.zeros_like(t))


def _statistics(x, see, n):
    mean = _kept(x, see).sum((1, 3)) / n
    d = _kept(x - mean[:, None, :, None], see)
    return mean, torch.rsqrt(d.square().sum((1, 3)) / n + _EPS)


def _plain_group_norm(s):
    x, see, n = _grouped(s, s["x"].float())
    mean, rstd = _statistics(x, see, n)
    side = (1, 1, s["groups"], -1)
    z = (x - mean[:, None, :, None]) * rstd[:, None, :, None] * s["weight"].float().view(side) + s["bias"].float().view(side)
    if s["activation"] == "relu":
        z = z.clamp(min=0.0)
    elif s["activation"] == "silu":
        z = z * torch.sigmoid(z)
    return {"y": _kept(z, see).view(s["x"].shape).to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_group_norm_backward(s):
    x, see, n = _grouped(s, s["x"].float())
    dt, side = s["x"].dtype, (1, 1, s["groups"], -1)
    g = s["g"].float().view(x.shape)
    rstd = s["rstd"][:, None, :, None]
    w = s["weight"].float().view(side)
    xh = (x - s["mean"][:, None, :, None]) * rstd
    if s["activation"]:
        z = xh * w + s["bias"].float().view(side)
        if s["activation"] == "relu":
            g = g * (z > 0)
        else:
            p = torch.sigmoid(z)
            g = g * p * (1 + z * (1 - p))
    g = _kept(g, see)
    u = g * w
    n = n if see is None else n.view(-1, 1, 1, 1)
    gx = rstd * (u - u.sum((1, 3), keepdim=True) / n - xh * ((u * xh).sum((1, 3), keepdim=True) / n))
    return {"x": _kept(gx, see).view(s["x"].shape).to(dt), "weight": (g * xh).sum((0, 1)).view(-1).to(dt),
            "bias": g.sum((0, 1)).view(-1).to(dt)}


def _order(s, t):
    """t [B, L, C] in the order of the recurrence, which is its own inverse."""
    if not s["reverse"]:
        return t
    if s["lens"] is None:
        return t.flip(1)
    i = torch.arange(s["L"], device="cuda").view(1, -1)
    n = s["lens"].long().view(-1, 1)
    at = torch.where(i < n, n - 1 - i, i)
    return torch.gather(t, 1, at.unsqueeze(2).expand(-1, -1, s["C"]))


def _in_length(s):
    if s["lens"] is None:
        return None
    return torch.arange(s["L"], device="cuda").view(1, -1, 1) < s["lens"].view(-1, 1, 1)


def _gates(s):
    """The factors a and the terms u of h' = a h + u, in the recurrence's order; (1, 0) past a sequence's length."""
    x, gate = _order(s, s["x"].float()), _order(s, s["gate"].float())
    a, b = torch.sigmoid(gate), torch.sigmoid(-gate)
    u, see = (b * x if s["blend"] else x), _in_length(s)
    if see is not None:
        a, u = torch.where(see, a, torch.ones_like(a)), _kept(u, see)
    return x, a, b, u, see


def _scan(a, h):
    """h[t] = a[t] h[t-1] + h[t] from nothing, over axis 1: spans of growing length are joined."""
    a, h, d = a.clone(), h.clone(), 1
    while d < a.shape[1]:
        h = torch.cat([h[:, :d], h[:, d:] + a[:, d:] * h[:, :-d]], 1)
        a = torch.cat([a[:, :d], a[:, d:] * a[:, :-d]], 1)
        d *= 2
    return h


def _plain_states(s, a, u):
    """The states after every position."""
    u = torch.cat([u[:, :1] + a[:, :1] * s["state"].unsqueeze(1), u[:, 1:]], 1)
    return _scan(a, u)


def _plain_recurrence(s):
    _, a, _, u, see = _gates(s)
    h = _plain_states(s, a, u)
    before = torch.cat([s["state"].unsqueeze(1), h[:, :-1]], 1)
    return {"y": _order(s, _kept(h, see)).to(s["x"].dtype), "last": h[:, -1].contiguous(),
            "states": before[:, ::_EVERY].contiguous()}


def _plain_recurrence_backward(s):
    x, a, b, u, see = _gates(s)
    h = _plain_states(s, a, u)
    before = torch.cat([s["state"].unsqueeze(1), h[:, :-1]], 1)
    g = _kept(_order(s, s["g"].float()), see)
    # r[t] = g[t] + a[t+1] r[t+1], the last one's from the last state's gradient
    g = torch.cat([g[:, :-1], g[:, -1:] + s["g_last"].unsqueeze(1)], 1)
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    r = _scan(after.flip(1), g.flip(1)).flip(1)
    gx, gg = (r * b, r * (before - x) * a * b) if s["blend"] else (r, r * before * a * b)
    dt = s["x"].dtype
    return {"x": _order(s, _kept(gx, see)).to(dt), "gate": _order(s, _kept(gg, see)).to(dt), "state": a[:, 0] * r[:, 0]}


# ---- one pass ----------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from deformable_convolution_amd import sequence
        if op in ("gn_fwd", "gn_bwd"):
            kw = dict(activation=s["activation"] or None, lens=s["lens"])
            if op == "gn_fwd":
                y, mean, rstd = sequence.group_norm(s["x"], s["groups"], s["weight"], s["bias"], eps=_EPS, with_stats=True, **kw)
                return {"y": y, "mean": mean, "rstd": rstd}
            return sequence.group_norm_backward(s["x"], s["groups"], s["g"], s["mean"], s["rstd"], s["weight"], s["bias"], **kw)
        kw = dict(lens=s["lens"], blend=s["blend"], reverse=s["reverse"])
        if op == "rec_fwd":
            y, last, states = sequence.gated_recurrence(s["x"], s["gate"], state=s["state"], with_states=True, **kw)
            return {"y": y, "last": last, "states": states}
        return sequence.gated_recurrence_backward(s["x"], s["gate"], s["states"], s["g"], grad_last=s["g_last"], **kw)
    if op == "gn_fwd":
        return _plain_group_norm(s)
    if op == "gn_bwd":
        return _plain_group_norm_backward(s)
    if op == "rec_fwd":
        return _plain_recurrence(s)
    return _plain_recurrence_backward(s)


# ---- work --------------------------------------------------------------------

def work(case):
    e, op, B, C = _SIZE[case["dtype"]], case["op"], case["B"], case["C"]
    n = max(1, case["S"] if op in ("gn_fwd", "gn_bwd") else case["L"])
    rows = B * n  # every position is written, those within the lengths are read
    seen = sum(_lengths(B, n)) if case["ragged"] else rows
    if op == "gn_fwd":
        return {"bytes": e * C * (seen + rows) + 2 * e * C + 8 * B * case["groups"], "flops": 10 * seen * C}
    if op == "gn_bwd":
        return {"bytes": e * C * (2 * seen + rows) + 4 * e * C + 8 * B * case["groups"], "flops": 24 * seen * C}
    states = 4 * B * C * (-(-n // _EVERY))
    if op == "rec_fwd":
        return {"bytes": e * C * (2 * seen + rows) + states + 8 * B * C, "flops": 10 * seen * C}
    return {"bytes": e * C * (3 * seen + 2 * rows) + states + 8 * B * C, "flops": 24 * seen * C}


# ---- 64 bits -----------------------------------------------------------------

def exact(case, seed):
    """The definitions in float64: sequence by sequence and group by group, position by position."""
    s = prepare(case, seed)
    op, f8, B, C = case["op"], torch.float64, case["B"], case["C"]
    if op in ("gn_fwd", "gn_bwd"):
        S, G = max(1, case["S"]), case["groups"]
        D = C // G
        x = s["x"].to(f8).reshape(B, S, C)
        w, b = s["weight"].to(f8), s["bias"].to(f8)
        lens = s["lens"].tolist() if s["lens"] is not None else None
        # one batch of equal lengths, or sequence by sequence
        parts = [(slice(0, B), S)] if lens is None else [(slice(i, i + 1), n) for i, n in enumerate(lens)]
        mean = torch.zeros((B, G), dtype=f8, device="cuda")
        rstd = torch.zeros_like(mean)
        out = torch.zeros((B, S, C), dtype=f8, device="cuda")
        gw, gb = torch.zeros(C, dtype=f8, device="cuda"), torch.zeros(C, dtype=f8, device="cuda")
        for at, n in parts:
            for k in range(G):
                c = slice(k * D, (k + 1) * D)
                v = x[at, :n, c]
                m = v.mean((1, 2))
                r = (v.var((1, 2), unbiased=False) + _EPS).pow(-0.5) if n * D > 1 else torch.full_like(m, _EPS ** -0.5)
                mean[at, k], rstd[at, k] = m, r
                xh = (v - m[:, None, None]) * r[:, None, None]
                z = xh * w[c] + b[c]
                if op == "gn_fwd":
                    if case["activation"] == "relu":
                        z = torch.where(z > 0, z, torch.zeros_like(z))
                    elif case["activation"] == "silu":
                        z = z / (1 + torch.exp(-z))
                    out[at, :n, c] = z
                    continue
                g = s["g"].to(f8).reshape(B, S, C)[at, :n, c]
                if case["activation"] == "relu":
                    g = torch.where(z > 0, g, torch.zeros_like(g))
                elif case["activation"] == "silu":
                    q = torch.exp(-z)
                    g = g * (1 + q + z * q) / (1 + q).square()
                gw[c] += (g * xh).sum((0, 1))
                gb[c] += g.sum((0, 1))
                u = g * w[c]
                out[at, :n, c] = (u - u.mean((1, 2), keepdim=True) - xh * (u * xh).mean((1, 2), keepdim=True)) * r[:, None, None]
        out = out.reshape(s["x"].shape)
        return {"y": out, "mean": mean, "rstd": rstd} if op == "gn_fwd" else {"x": out, "weight": gw, "bias": gb}
    L = case["L"]
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), L, dtype=torch.long, device="cuda")
    batch = torch.arange(B, device="cuda")
    steps = torch.arange(L, device="cuda").view(L, 1).expand(L, B)
    at = (lens - 1 - steps).clamp(min=0) if case["reverse"] else steps  # [L, B]: where step i of each sequence stands
    on = (steps < lens).unsqueeze(2)
    h = s["state"].to(f8)
    before = torch.empty((L, B, C), dtype=f8, device="cuda")
    y = torch.zeros((B, L, C), dtype=f8, device="cuda")

    def factors(i):
        x, gate = s["x"][batch, at[i]].to(f8), s["gate"][batch, at[i]].to(f8)
        keep = 1 / (1 + torch.exp(-gate))
        return x, keep, 1 / (1 + torch.exp(gate))

    def put(t, i, v):
        """Row i of each sequence that is that long; the others' rows stay."""
        t[batch, at[i]] = torch.where(on[i], v, t[batch, at[i]])

    for i in range(L):
        before[i] = h
        x, keep, drop = factors(i)
        h = torch.where(on[i], keep * h + (drop * x if case["blend"] else x), h)
        if op == "rec_fwd":
            put(y, i, h)
    if op == "rec_fwd":
        return {"y": y, "last": h, "states": before[::_EVERY].transpose(0, 1).contiguous()}
    r = s["g_last"].to(f8)  # the gradient of the state after step i
    gx, gg = y, torch.zeros_like(y)
    for i in range(L - 1, -1, -1):
        x, keep, drop = factors(i)
        r = torch.where(on[i], r + s["g"][batch, at[i]].to(f8), r)
        put(gx, i, r * drop if case["blend"] else r)
        put(gg, i, r * ((before[i] - x) if case["blend"] else before[i]) * keep * drop)
        r = torch.where(on[i], r * keep, r)
    return {"x": gx, "gate": gg, "state": r}
