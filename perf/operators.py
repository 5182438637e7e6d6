"""The sequence operators' measured cases and their plain forms.

Layer norm over the channel axis, rotary positions with several axes,
attention and attention's gradients: what a sequence or image model puts next
to a deformable convolution.  Sizes follow the package's own workloads (the
layer's 16 x 512 x 128, the long sequence 8 x 256 x 16384, the depthwise
16 x 512 x 4096, the strided layer's 32 x 1024 x 1024 output, 64 x 64 and
28 x 28 images).

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


# ---- cases -------------------------------------------------------------------

def _ln(op, B, C, L, dtype):
    """L = 0: rows [B, C]; else channels first [B, C, L]."""
    return {"op": op, "B": B, "C": C, "L": L, "dtype": dtype}


def _rot(B, L, Hq, Hkv, D, sections, dtype, inverse=False, interleaved=False):
    return {"op": "rotary", "B": B, "L": L, "Hq": Hq, "Hkv": Hkv, "D": D, "sections": sections, "dtype": dtype,
            "inverse": inverse, "interleaved": interleaved}


def _att(op, B, Lq, Lk, Hq, Hkv, D, dtype, causal=False, window=0, ragged=False):
    """ragged: key lengths from a quarter of Lk up to Lk, the queries the last of each sequence's keys if causal."""
    return {"op": op, "B": B, "Lq": Lq, "Lk": Lk, "Hq": Hq, "Hkv": Hkv, "D": D, "dtype": dtype, "causal": causal,
            "window": window, "ragged": ragged}


def listed():
    return [
        # one new position of each of 16 sequences, ahead of a projection: latency
        dict(_ln("ln_fwd", 16, 512, 0, "f32"), name="ln_fwd_step"),
        # the long bf16 sequence, normalised between two convolutions
        dict(_ln("ln_fwd", 8, 256, 16384, "bf16"), name="ln_fwd_long"),
        # training on the strided layer's output taken as 32 x 1024 tokens of 1024 channels
        dict(_ln("ln_bwd", 32768, 1024, 0, "bf16"), name="ln_bwd_tokens"),
        # training, channels first, at the depthwise layer's size
        dict(_ln("ln_bwd", 16, 512, 4092, "f32"), name="ln_bwd_channels"),
        # one new position of each of 16 sequences, shared key heads
        dict(_rot(16, 1, 8, 2, 128, "64", "bf16"), name="rotary_step"),
        # four 28 x 28 frames and a few text positions of two clips: time, height and width
        dict(_rot(2, 3147, 8, 2, 128, "16,24,24", "bf16"), name="rotary_video"),
        # gradients of 64 x 64 images' rotated heads: rows and columns
        dict(_rot(8, 4096, 8, 8, 64, "16,16", "f32", inverse=True, interleaved=True), name="rotary_image_bwd"),
        # one new position of each of 16 sequences over caches of up to 16384
        dict(_att("att_fwd", 16, 1, 16384, 8, 2, 128, "bf16", causal=True, ragged=True), name="att_step"),
        # the layer's 83 output positions, 512 channels in 8 heads, full precision
        dict(_att("att_fwd", 16, 83, 83, 8, 8, 64, "f32"), name="att_fwd_layer"),
        # 64 x 64 images as 4096 positions, 512 channels in 8 heads
        dict(_att("att_fwd", 8, 4096, 4096, 8, 8, 64, "bf16"), name="att_fwd_image"),
        # training on 128 positions of padded batches, full precision
        dict(_att("att_bwd", 16, 128, 128, 8, 8, 64, "f32", ragged=True), name="att_bwd_layer"),
        # causal training on 4096 positions, 1024 channels in 8 heads over 2 key heads
        dict(_att("att_bwd", 4, 4096, 4096, 8, 2, 128, "bf16", causal=True), name="att_bwd_causal"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _keep(n):
    """Not 3072: a neighbour of it."""
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "rotary", "att_fwd", "att_step", "att_bwd"])
    dtype = rng.choice(["f32", "bf16"])
    if op in ("ln_fwd", "ln_bwd"):
        C = _keep(_log(rng, 32, 2048))
        if rng.random() < 0.5:
            return _ln(op, _keep(_log(rng, 1, max(1, (1 << 25) // C))), C, 0, dtype)
        L = _keep(_log(rng, 16, 16384))
        return _ln(op, _keep(_log(rng, 1, max(1, min(64, (1 << 25) // (C * L))))), C, L, dtype)
    D = rng.choice([32, 64, 64, 80, 128, 128])
    Hkv = rng.choice([1, 2, 4])
    Hq = Hkv * rng.choice([1, 1, 2, 4])
    if op == "rotary":
        R = D // 2
        a = R // 4 + rng.randrange(R // 4)
        sections = rng.choice(["%d" % R, "%d,%d" % (a, R - a), "%d,%d,%d" % (a, (R - a) // 2, R - a - (R - a) // 2)])
        L = _keep(_log(rng, 1, 16384))
        B = _log(rng, 1, max(1, min(32, (1 << 24) // (L * (Hq + Hkv) * D))))
        return _rot(B, L, Hq, Hkv, D, sections, dtype, rng.random() < 0.5, rng.random() < 0.5)
    if op == "att_step":
        Lk = _keep(_log(rng, 64, 16384))
        return _att("att_fwd", _log(rng, 1, 16), rng.choice([1, 1, 1, 2, 5]), Lk, Hq, Hkv, D, dtype, causal=True,
                    window=rng.choice([0, 0, 1024]), ragged=True)
    # a full-precision pass has a sixteenth of the matrix rate: shorter sequences keep it within the largest case's time
    L = _keep(_log(rng, 17, 4096 if dtype == "bf16" else 2048))
    Lk = L if rng.random() < 0.7 else _keep(_log(rng, 17, L))
    causal = rng.random() < 0.5
    B = _log(rng, 1, max(1, min(32, (1 << (26 if dtype == "bf16" else 24)) // (L * Lk * Hq // 4))))
    return _att(op, B, L, Lk, Hq, Hkv, D, dtype, causal, rng.choice([0, 0, 0, 257]), rng.random() < 0.3)


# ---- inputs ------------------------------------------------------------------

def _lens(case, gen):
    """The ragged key lengths: evenly spread, dealt out by the seed."""
    B, Lk = case["B"], case["Lk"]
    lo = max(1, Lk // 4)
    n = [lo + (Lk - lo) * (b + 1) // B for b in range(B)]
    order = torch.randperm(B, generator=gen, device=gen.device)
    return torch.tensor(n, dtype=torch.int32, device=gen.device)[order].contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    op = case["op"]
    s = dict(case)
    if op in ("ln_fwd", "ln_bwd"):
        shape = (case["B"], case["C"], case["L"]) if case["L"] else (case["B"], case["C"])
        s["x"] = (torch.randn(shape, generator=gen, device="cuda") * 1.5 + 0.25).to(dt)
        s["weight"] = (1 + 0.2 * torch.randn(case["C"], generator=gen, device="cuda")).to(dt)
        s["bias"] = (0.2 * torch.randn(case["C"], generator=gen, device="cuda")).to(dt)
        if op == "ln_bwd":
            s["g"] = randn(*shape)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"].unsqueeze(1)).square().mean(1) + _EPS)
        return s
    B, D, Hq, Hkv = case["B"], case["D"], case["Hq"], case["Hkv"]
    if op == "rotary":
        L = case["L"]
        counts = [int(v) for v in case["sections"].split(",")]
        R, A, P = sum(counts), len(counts), max(L, 64) if len(counts) == 1 else 4096
        angle = torch.arange(P, device="cuda", dtype=torch.float64).unsqueeze(1) * torch.pow(
            10000.0, -torch.arange(R, device="cuda", dtype=torch.float64) / R)
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        if A == 1:  # consecutive positions from each sequence's own start
            first = torch.randint(0, P - L + 1, (B, 1, 1), generator=gen, device="cuda")
            s["positions"] = (first + torch.arange(L, device="cuda").view(1, L, 1)).int()
        else:
            s["positions"] = torch.randint(0, P, (B, L, A), generator=gen, device="cuda").int()
        s["counts"] = counts
        # the heads of one product: queries, then keys
        both = randn(B, L, Hq + Hkv, D)
        s["q"], s["k"] = both[:, :, :Hq], both[:, :, Hq:]
        return s
    Lq, Lk = case["Lq"], case["Lk"]
    s["q"] = randn(B, Lq, Hq, D)
    s["k"] = randn(B, Lk, Hkv, D)
    s["v"] = randn(B, Lk, Hkv, D)
    s["kv_lens"] = _lens(case, gen) if case["ragged"] else None
    s["q_start"] = s["kv_lens"] - Lq if case["ragged"] and case["causal"] else None
    if op == "att_bwd":
        s["g"] = randn(B, Lq, Hq, D)
        s["out"], s["lse"] = _plain_attention(s)
    return s


# ---- plain forms -------------------------------------------------------------

def _plain_layer_norm(s):
    x = s["x"].float()
    side = (1, -1, 1) if s["L"] else (1, -1)
    mean = x.mean(1)
    d = x - mean.unsqueeze(1)
    rstd = torch.rsqrt(d.square().mean(1) + _EPS)
    y = d * rstd.unsqueeze(1) * s["weight"].float().view(side) + s["bias"].float().view(side)
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_layer_norm_backward(s):
    x, g = s["x"].float(), s["g"].float()
    side, rest = ((1, -1, 1), (0, 2)) if s["L"] else ((1, -1), (0,))
    rstd = s["rstd"].unsqueeze(1)
    xh = (x - s["mean"].unsqueeze(1)) * rstd
    gh = g * s["weight"].float().view(side)
    gx = rstd * (gh - gh.mean(1, keepdim=True) - xh * (gh * xh).mean(1, keepdim=True))
    dt = s["x"].dtype
    return {"x": gx.to(dt), "weight": (g * xh).sum(rest).to(dt), "bias": g.sum(rest).to(dt)}


def _plain_rotary(s):
    counts, R = s["counts"], sum(s["counts"])
    axis = torch.repeat_interleave(torch.arange(len(counts), device="cuda"), torch.tensor(counts, device="cuda"),
                                   output_size=R)
    row = s["positions"].long()[:, :, axis]  # [B, L, R]
    pair = torch.arange(R, device="cuda")
    c, d = s["cos"][row, pair].unsqueeze(2), s["sin"][row, pair].unsqueeze(2)
    if s["inverse"]:
        d = -d

    def turn(x):
        f = x.float()
        a, b = (f[..., 0:2 * R:2], f[..., 1:2 * R:2]) if s["interleaved"] else (f[..., :R], f[..., R:2 * R])
        y = [a * c - b * d, a * d + b * c]
        return (torch.stack(y, -1).flatten(-2) if s["interleaved"] else torch.cat(y, -1)).to(x.dtype)

    return {"q": turn(s["q"]), "k": turn(s["k"])}


def _visible(s):
    """[B, 1, Lq, Lk] truth values, or None where everything is visible."""
    B, Lq, Lk = s["B"], s["Lq"], s["Lk"]
    if s["kv_lens"] is None and not s["causal"] and not s["window"]:
        return None
    j = torch.arange(Lk, device="cuda").view(1, 1, 1, Lk)
    start = s["q_start"].long().view(B, 1, 1, 1) if s["q_start"] is not None else Lk - Lq
    p = start + torch.arange(Lq, device="cuda").view(1, 1, Lq, 1)
    see = torch.ones((1, 1, 1, 1), dtype=torch.bool, device="cuda")
    if s["kv_lens"] is not None:
        see = see & (j < s["kv_lens"].long().view(B, 1, 1, 1))
    if s["causal"]:
        see = see & (j <= p)
    if s["window"]:
        see = see & (p - j < s["window"]) & (j - p < s["window"])
    return see


def _heads(x, times=1):
    """[B, L, H, D] as float32 [B, H * times, L, D], each head repeated."""
    x = x.float().transpose(1, 2)
    return (x.repeat_interleave(times, 1) if times > 1 else x).contiguous()


def _scores(s):
    group = s["Hq"] // s["Hkv"]
    q, k, v = _heads(s["q"]), _heads(s["k"], group), _heads(s["v"], group)
    S = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(s["D"]))
    see = _visible(s)
    if see is not None:
        S = S.masked_fill_(~see, -math.inf)
    top = S.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    P = S.sub_(top).exp_()
    total = P.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)
    return q, k, v, P, total, lse


def _plain_attention(s):
    q, k, v, P, total, lse = _scores(s)
    out = torch.matmul(P, v) / torch.where(total == 0, torch.ones_like(total), total)
    return out.transpose(1, 2).contiguous().to(s["q"].dtype), lse


def _plain_attention_backward(s):
    q, k, v, P, total, _ = _scores(s)
    P = P.div_(torch.where(total == 0, torch.ones_like(total), total))
    g = _heads(s["g"])
    group, B, D, dt = s["Hq"] // s["Hkv"], s["B"], s["D"], s["q"].dtype
    gv = torch.matmul(P.transpose(2, 3).contiguous(), g)
    dP = torch.matmul(g, v.transpose(2, 3).contiguous())
    delta = (P * dP).sum(-1, keepdim=True)
    dS = dP.sub_(delta).mul_(P).mul_(1.0 / math.sqrt(D))
    gq = torch.matmul(dS, k)
    gk = torch.matmul(dS.transpose(2, 3).contiguous(), q)
    shared = lambda t: t.view(B, s["Hkv"], group, s["Lk"], D).sum(2).transpose(1, 2).contiguous().to(dt)  # noqa: E731
    return {"q": gq.transpose(1, 2).contiguous().to(dt), "k": shared(gk), "v": shared(gv)}


# ---- one pass ----------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        from deformable_convolution_amd import sequence
        if op == "ln_fwd":
            y, mean, rstd = sequence.layer_norm(s["x"], s["weight"], s["bias"], eps=_EPS, with_stats=True)
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "ln_bwd":
            return sequence.layer_norm_backward(s["x"], s["g"], s["mean"], s["rstd"], s["weight"])
        if op == "rotary":
            q, k = sequence.rotary(s["q"], s["k"], s["cos"], s["sin"], s["positions"], s["counts"],
                                   interleaved=s["interleaved"], inverse=s["inverse"])
            return {"q": q, "k": k}
        kw = dict(causal=s["causal"], window=s["window"], kv_lens=s["kv_lens"], q_start=s["q_start"])
        if op == "att_fwd":
            out, lse = sequence.attention(s["q"], s["k"], s["v"], with_lse=True, **kw)
            return {"out": out, "lse": lse}
        return sequence.attention_backward(s["q"], s["k"], s["v"], s["out"], s["lse"], s["g"], **kw)
    if op == "ln_fwd":
        return _plain_layer_norm(s)
    if op == "ln_bwd":
        return _plain_layer_norm_backward(s)
    if op == "rotary":
        return _plain_rotary(s)
    if op == "att_fwd":
        out, lse = _plain_attention(s)
        return {"out": out, "lse": lse}
    return _plain_attention_backward(s)


# ---- work --------------------------------------------------------------------

def _seen(case):
    """Visible (query, key) pairs of one head, over the batch, and the keys that any query sees."""
    B, Lq, Lk, w = case["B"], case["Lq"], case["Lk"], case["window"]
    lo = max(1, Lk // 4)
    pairs = keys = 0
    for b in range(B):
        n = lo + (Lk - lo) * (b + 1) // B if case["ragged"] else Lk
        start = n - Lq if case["ragged"] and case["causal"] else Lk - Lq
        if not case["causal"] and not w:
            pairs += Lq * n
            keys += n
            continue
        first, last = Lk, 0
        for i in range(Lq):
            p = start + i
            hi = min(n, p + 1) if case["causal"] else min(n, p + w)
            at = max(0, p - w + 1) if w else 0
            if hi > at:
                pairs += hi - at
                first, last = min(first, at), max(last, hi)
        keys += max(0, last - first)
    return pairs, keys


def work(case):
    e, op = _SIZE[case["dtype"]], case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        C, rows = case["C"], case["B"] * max(1, case["L"])
        if op == "ln_fwd":
            return {"bytes": 2 * e * rows * C + 2 * e * C + 8 * rows, "flops": 7 * rows * C}
        return {"bytes": 3 * e * rows * C + 3 * e * C + 8 * rows, "flops": 14 * rows * C}
    B, D, Hq, Hkv = case["B"], case["D"], case["Hq"], case["Hkv"]
    if op == "rotary":
        R, A = D // 2, len(case["sections"].split(","))
        n = B * case["L"]
        table = 8 * R * (min(n, max(case["L"], 64)) if A == 1 else min(n * A, 4096))
        return {"bytes": 2 * e * n * (Hq + Hkv) * D + 4 * n * A + table, "flops": 3 * n * (Hq + Hkv) * D}
    pairs, keys = _seen(case)
    rows = B * case["Lq"] * Hq
    if op == "att_fwd":
        return {"bytes": 2 * e * rows * D + 4 * rows + 2 * e * keys * Hkv * D, "flops": 4 * pairs * Hq * D}
    # reads q, out, g, k, v and writes three gradients, those of unseen keys too
    return {"bytes": 4 * e * rows * D + 4 * rows + 2 * e * keys * Hkv * D + 2 * e * B * case["Lk"] * Hkv * D,
            "flops": 10 * pairs * Hq * D}


# ---- 64 bits -----------------------------------------------------------------

def exact(case, seed):
    """The definitions in float64, one position of the sum after another kept apart from the plain forms."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64
    if op in ("ln_fwd", "ln_bwd"):
        rows = s["x"].to(f8)
        rows = rows.transpose(1, 2) if case["L"] else rows  # channels last
        mean = rows.sum(-1) / case["C"]
        var = (rows * rows).sum(-1) / case["C"] - mean * mean
        rstd = (var + _EPS).pow(-0.5)
        xh = (rows - mean[..., None]) * rstd[..., None]
        w = s["weight"].to(f8)
        back = lambda t: t.transpose(1, 2) if case["L"] else t  # noqa: E731
        if op == "ln_fwd":
            return {"y": back(xh * w + s["bias"].to(f8)), "mean": mean, "rstd": rstd}
        g = s["g"].to(f8)
        g = g.transpose(1, 2) if case["L"] else g
        lead = tuple(range(g.dim() - 1))
        u = g * w
        gx = (u - (u.sum(-1, keepdim=True) + xh * (u * xh).sum(-1, keepdim=True)) / case["C"]) * rstd[..., None]
        return {"x": back(gx), "weight": (g * xh).sum(lead), "bias": g.sum(lead)}
    if op == "rotary":
        R, pos = sum(s["counts"]), s["positions"].long()
        parts, at = [], 0
        for a, n in enumerate(s["counts"]):  # the turn of each pair as a complex number
            rows = pos[:, :, a]
            parts.append(torch.complex(s["cos"].to(f8)[rows, at:at + n], s["sin"].to(f8)[rows, at:at + n]))
            at += n
        turn = torch.cat(parts, -1).unsqueeze(2)
        turn = turn.conj() if case["inverse"] else turn

        def rotated(x):
            x = x.to(f8)
            x = x.unflatten(-1, (R, 2)) if case["interleaved"] else x.unflatten(-1, (2, R)).transpose(-1, -2)
            y = torch.view_as_real(torch.view_as_complex(x.contiguous()) * turn)
            return (y if case["interleaved"] else y.transpose(-1, -2)).flatten(-2).contiguous()

        return {"q": rotated(s["q"]), "k": rotated(s["k"])}
    B, Lq, Lk, Hq, Hkv, D = (case[k] for k in ("B", "Lq", "Lk", "Hq", "Hkv", "D"))
    group = Hq // Hkv
    got = {k: [] for k in ("out", "lse", "q", "k", "v")}
    for b in range(B):
        n = int(s["kv_lens"][b]) if s["kv_lens"] is not None else Lk
        p = torch.arange(Lq, device="cuda") + (int(s["q_start"][b]) if s["q_start"] is not None else Lk - Lq)
        away = p.view(Lq, 1) - torch.arange(n, device="cuda").view(1, n)  # the key's distance behind the query
        hide = torch.zeros((Lq, n), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hide |= away < 0
        if case["window"]:
            hide |= away.abs() >= case["window"]
        empty = hide.all(1) if n else torch.ones(Lq, dtype=torch.bool, device="cuda")
        out = torch.zeros((Lq, Hq, D), dtype=f8, device="cuda")
        lse = torch.full((Hq, Lq), -math.inf, dtype=f8, device="cuda")
        gq = torch.zeros((Lq, Hq, D), dtype=f8, device="cuda")
        gk = torch.zeros((Lk, Hkv, D), dtype=f8, device="cuda")
        gv = torch.zeros((Lk, Hkv, D), dtype=f8, device="cuda")
        for h in range(Hq):
            q, k, v = s["q"][b, :, h].to(f8), s["k"][b, :n, h // group].to(f8), s["v"][b, :n, h // group].to(f8)
            z = (q @ k.t().contiguous()) / math.sqrt(D)
            z[hide] = -math.inf
            lse[h] = torch.logsumexp(z, 1)
            P = torch.exp(z - torch.where(empty, torch.zeros_like(lse[h]), lse[h])[:, None])
            o = P @ v
            if op == "att_fwd":
                out[:, h] = o
                continue
            g = s["g"][b, :, h].to(f8)
            gv[:n, h // group] += P.t().contiguous() @ g
            W = P * (g @ v.t().contiguous() - (g * o).sum(1, keepdim=True)) / math.sqrt(D)
            gq[:, h] = W @ k
            gk[:n, h // group] += W.t().contiguous() @ q
        for key, t in zip(("out", "lse", "q", "k", "v"), (out, lse, gq, gk, gv)):
            got[key].append(t)
    if op == "att_fwd":
        return {"out": torch.stack(got["out"]), "lse": torch.stack(got["lse"])}
    return {key: torch.stack(got[key]) for key in ("q", "k", "v")}
