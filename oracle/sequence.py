"""Plain double-precision forms of the sequence operators (layer norm over
axis 1, rotary positions, attention) and their gradients, written from the
formulas with torch's elementary operations in float64.  Test infrastructure
only; runs on the device its inputs are on.

The ``*_bound`` functions give elementwise bounds of the rounding errors
that an implementation may make which keeps sums and statistics in 32 bits
and rounds each result (and, in bf16, the probabilities and score gradients)
once; ``u`` is the unit roundoff 2^-24 (fp32) or 2^-8 (bf16).
"""
import math

import torch

F8 = torch.float64


def unit(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24


def _side(x):
    return (1, -1) + (1,) * (x.dim() - 2)


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    x = x.to(F8)
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean) ** 2).mean(1, keepdim=True).add(eps) ** -0.5
    y = (x - mean) * rstd
    if weight is not None:
        y = y * weight.to(F8).view(_side(x))
    if bias is not None:
        y = y + bias.to(F8).view(_side(x))
    return y, mean.squeeze(1), rstd.squeeze(1)


def layer_norm_backward(x, g, weight=None, eps=1e-5):
    _, mean, rstd = layer_norm(x, eps=eps)
    mean, rstd = mean.unsqueeze(1), rstd.unsqueeze(1)
    x, g = x.to(F8), g.to(F8)
    xh = (x - mean) * rstd
    u = g if weight is None else g * weight.to(F8).view(_side(x))
    gx = rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True))
    rest = [0] + list(range(2, x.dim()))
    return {"x": gx, "weight": (g * xh).sum(rest), "bias": g.sum(rest)}


def rotary(x, cos, sin, positions, sections, interleaved=False, inverse=False):
    x = x.to(F8)
    R, P = sum(sections), cos.shape[0]
    y = x.clone()
    positions = positions.long().clamp(0, P - 1).expand(x.shape[0], -1, -1)
    i = 0
    for axis, n in enumerate(sections):
        for _ in range(n):
            p = positions[:, :, axis]
            c, s = cos.to(F8)[p, i].unsqueeze(-1), sin.to(F8)[p, i].unsqueeze(-1)
            if inverse:
                s = -s
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, R + i)
            y[..., a] = x[..., a] * c - x[..., b] * s
            y[..., b] = x[..., a] * s + x[..., b] * c
            i += 1
    return y


def visible(B, Lq, Lk, causal=False, window=0, kv_lens=None, q_start=None, device=None):
    """[B, Lq, Lk]: which keys each query sees."""
    j = torch.arange(Lk, device=device).view(1, 1, Lk)
    start = torch.full((B, 1, 1), Lk - Lq, device=device) if q_start is None else q_start.long().view(B, 1, 1)
    p = start + torch.arange(Lq, device=device).view(1, Lq, 1)
    see = torch.ones((B, Lq, Lk), dtype=torch.bool, device=device)
    if kv_lens is not None:
        see &= j < kv_lens.long().view(B, 1, 1)
    if causal:
        see &= j <= p
    if window:
        see &= (p - j).abs() < window
    return see


def _bhld(t, times=1):
    t = t.to(F8).transpose(1, 2)
    return t.repeat_interleave(times, 1).contiguous()


def _scores(q, k, v, see, scale):
    G = q.shape[2] // k.shape[2]
    used = see.any(1)[:, :, None, None]  # keys that nobody sees are not looked at
    zero = torch.zeros((), dtype=F8, device=k.device)
    k, v = torch.where(used, k.to(F8), zero), torch.where(used, v.to(F8), zero)
    Q, K, V = _bhld(q), _bhld(k, G), _bhld(v, G)
    S = torch.matmul(Q, K.transpose(2, 3).contiguous()) * scale
    S = torch.where(see.unsqueeze(1), S, torch.full_like(S, -math.inf))
    if S.shape[-1]:
        lse = torch.logsumexp(S, -1)
    else:
        lse = torch.full(S.shape[:-1], -math.inf, dtype=F8, device=S.device)
    P = torch.exp(S - torch.where(lse == -math.inf, torch.zeros_like(lse), lse).unsqueeze(-1))
    return Q, K, V, S, P, lse


def attention(q, k, v, scale=None, **mask):
    """out [B, Lq, Hq, D], lse [B, Hq, Lq] and the bound of out's error per unit
    roundoff of the probabilities, sum_j P |v|, in out's layout."""
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    see = visible(q.shape[0], q.shape[1], k.shape[1], device=q.device, **mask)
    _, _, V, _, P, lse = _scores(q, k, v, see, scale)
    back = lambda t: t.transpose(1, 2).contiguous()  # noqa: E731
    return back(P @ V), lse, back(P @ V.abs())


def attention_backward(q, k, v, g, scale=None, storage=torch.float32, **mask):
    """Gradients {q, k, v} and, for each, the bound of an implementation's error."""
    scale = 1 / math.sqrt(q.shape[3]) if scale is None else scale
    B, Lq, Hq, D = q.shape
    Hkv, Lk = k.shape[2], k.shape[1]
    see = visible(B, Lq, Lk, device=q.device, **mask)
    Q, K, V, S, P, _ = _scores(q, k, v, see, scale)
    g = _bhld(g)
    out = P @ V
    t = lambda a: a.transpose(2, 3).contiguous()  # noqa: E731
    dP = g @ t(V)
    delta = (g * out).sum(-1, keepdim=True)
    dS = P * (dP - delta)
    # What an implementation holds instead: P within ur (relative) of rounding
    # plus 64 u32 of the score's and exponential's own rounding; dP and delta
    # within 64 u32 of their absolute sums, delta also within ur of out's
    # rounding; dS rounded by ur.
    ur, u32 = unit(storage), 2.0 ** -24
    up = (ur if storage == torch.bfloat16 else 0.0) + 64 * u32
    dabs = (g.abs() * out.abs()).sum(-1, keepdim=True)
    e_p = up * P
    e_ds = up * dS.abs() + P * (64 * u32 * (g.abs() @ t(V.abs()) + dabs) + ur * dabs)
    shared = lambda a: a.reshape(B, Hkv, Hq // Hkv, Lk, D).sum(2).transpose(1, 2)  # noqa: E731
    grads = {"q": (scale * (dS @ K)).transpose(1, 2), "k": shared(scale * (t(dS) @ Q)), "v": shared(t(P) @ g)}
    more = 64 * u32
    bound = {"q": (scale * (e_ds @ K.abs() + more * (dS.abs() @ K.abs()))).transpose(1, 2),
             "k": shared(scale * (t(e_ds) @ Q.abs() + more * (t(dS.abs()) @ Q.abs()))),
             "v": shared(t(e_p) @ g.abs() + more * (t(P) @ g.abs()))}
    for n in grads:  # the result's own rounding
        bound[n] = bound[n] + ur * grads[n].abs()
    return grads, bound
