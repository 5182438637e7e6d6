"""Plain double-precision forms of group norm with an activation (channels
last) and of the gated linear recurrence, and their gradients, written from
the formulas.  Test infrastructure only; results are on the CPU.

The recurrence's ``*_bound`` values are elementwise bounds of the rounding
errors of an implementation that holds states in 32 bits: see
``gated_recurrence``.
"""
import torch

F8 = torch.float64
U32 = 2.0 ** -24


def _f8(t):
    return None if t is None else t.detach().cpu().to(F8)


def _lengths(lens, B, n):
    return [n] * B if lens is None else [min(max(int(v), 0), n) for v in lens.tolist()]


def _act(z, activation):
    """The activation and its derivative."""
    if activation == "relu":
        return z.clamp(min=0), (z > 0).to(F8)
    if activation == "silu":
        p = 1 / (1 + torch.exp(-z))
        return z * p, p * (1 + z * (1 - p))
    return z, torch.ones_like(z)


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, activation=None, lens=None, g=None):
    """y, mean, rstd; with g (grad_out) also the gradients {x, weight, bias}, and
    what bounds of rounding errors are made of, each of x's shape: xh, z, u =
    g act'(z) weight, and the absolute means of u and u xh over the group."""
    shape, C = x.shape, x.shape[-1]
    B, D = shape[0], C // groups
    x = _f8(x).reshape(B, -1, groups, D)
    S = x.shape[1]
    w = torch.ones(C, dtype=F8) if weight is None else _f8(weight)
    b = torch.zeros(C, dtype=F8) if bias is None else _f8(bias)
    w, b = w.view(groups, D), b.view(groups, D)
    mean, rstd = torch.zeros((B, groups), dtype=F8), torch.zeros((B, groups), dtype=F8)
    names = ("y", "xh", "z", "u", "gx", "au", "aux", "gz", "r")
    full = {n: torch.zeros_like(x) for n in names}
    gw, gb = torch.zeros((groups, D), dtype=F8), torch.zeros((groups, D), dtype=F8)
    for i, n in enumerate(_lengths(lens, B, S)):
        if n == 0:
            continue
        v = x[i, :n]
        m = v.mean((0, 2))
        r = ((v - m[None, :, None]) ** 2).mean((0, 2)).add(eps) ** -0.5
        mean[i], rstd[i] = m, r
        xh = (v - m[None, :, None]) * r[None, :, None]
        z = xh * w + b
        y, dy = _act(z, activation)
        full["y"][i, :n], full["xh"][i, :n], full["z"][i, :n] = y, xh, z
        full["r"][i, :n] = r[None, :, None]
        if g is not None:
            gz = _f8(g).reshape(x.shape)[i, :n] * dy
            u = gz * w
            gw += (gz * xh).sum(0)
            gb += gz.sum(0)
            full["gx"][i, :n] = r[None, :, None] * (u - u.mean((0, 2), keepdim=True) - xh * (u * xh).mean((0, 2), keepdim=True))
            full["u"][i, :n], full["gz"][i, :n] = u, gz
            full["au"][i, :n] = u.abs().mean((0, 2), keepdim=True)
            full["aux"][i, :n] = (u * xh).abs().mean((0, 2), keepdim=True)
    full = {n: t.reshape(shape) for n, t in full.items()}
    if g is None:
        return full["y"], mean, rstd
    return full["y"], mean, rstd, {"x": full["gx"], "weight": gw.view(C), "bias": gb.view(C)}, full


def gated_recurrence(x, gate, state=None, lens=None, blend=False, reverse=False, g=None, g_last=None):
    """A dict of y, last, states (ahead of every 64th position) and with g also
    the gradients gx, ggate, gstate; for each value ``name`` also
    ``name + "_bound"``, a bound of the error of 32-bit arithmetic:

    sigmoid(z) and 1 - it are off by k u, u = 2^-24, k = 10 + |z| relative (the
    exponential's argument |z| u, the exponential and the reciprocal two u each,
    three further roundings, and two for each product that a factor enters).
    A state's error then follows e' = a (e + k u S) + k u |term|, S the sum of the
    absolute values that make it up; a state that is put together from parts of
    the sequence has up to 64 further roundings of S."""
    x, gate, g, g_last, state = (_f8(t) for t in (x, gate, g, g_last, state))
    B, L, C = x.shape
    lens = _lengths(lens, B, L)
    back = g is not None
    kept = -(-L // 64)
    out = {n: torch.zeros((B, L, C), dtype=F8) for n in ("y", "gx", "ggate")}
    out.update(last=torch.zeros((B, C), dtype=F8), gstate=torch.zeros((B, C), dtype=F8), states=torch.zeros((B, kept, C), dtype=F8))
    out.update({n + "_bound": torch.zeros_like(t) for n, t in out.items()})
    JOIN = 64
    for b, n in enumerate(lens):
        order = [n - 1 - s if reverse else s for s in range(n)]
        h = state[b].clone() if state is not None else torch.zeros(C, dtype=F8)
        S, e = h.abs(), torch.zeros(C, dtype=F8)
        ahead = []
        a = 1 / (1 + torch.exp(-gate[b, :n]))
        q = 1 / (1 + torch.exp(gate[b, :n]))
        k = 10 + torch.where(torch.isinf(gate[b, :n]), torch.zeros_like(gate[b, :n]), gate[b, :n].abs())
        for s in range(L):
            if s % 64 == 0:
                out["states"][b, s // 64], out["states_bound"][b, s // 64] = h, U32 * (e + JOIN * S)
            if s >= n:
                continue
            t = order[s]
            ahead.append((h, e + JOIN * S))
            u = q[t] * x[b, t] if blend else x[b, t]
            h = a[t] * h + u
            e = a[t] * (e + k[t] * S) + k[t] * u.abs()
            S = a[t] * S + u.abs()
            out["y"][b, t], out["y_bound"][b, t] = h, U32 * (e + JOIN * S)
        out["last"][b], out["last_bound"][b] = h, U32 * (e + JOIN * S)
        if not back:
            continue
        m = g_last[b].clone() if g_last is not None else torch.zeros(C, dtype=F8)
        S, e = m.abs(), torch.zeros(C, dtype=F8)  # of m = a r, the gradient of the state ahead
        for s in range(n - 1, -1, -1):
            t = order[s]
            r, Sr = m + g[b, t], S + g[b, t].abs()
            er = e + JOIN * Sr
            h, eh = ahead[s]
            d = h - x[b, t] if blend else h
            ed = eh + h.abs() + x[b, t].abs()
            out["gx"][b, t] = r * q[t] if blend else r
            out["gx_bound"][b, t] = U32 * (er + k[t] * r.abs()) * (q[t] if blend else 1.0)
            out["ggate"][b, t] = r * d * a[t] * q[t]
            out["ggate_bound"][b, t] = U32 * a[t] * q[t] * (er * d.abs() + r.abs() * ed + 2 * k[t] * (r * d).abs())
            m = a[t] * r
            e = a[t] * (e + k[t] * Sr)
            S = a[t] * Sr
        out["gstate"][b], out["gstate_bound"][b] = m, U32 * (e + JOIN * S)
    return out
