"""The plain forms of oracle/block.py against torch's own operators, autograd
and differences, on the CPU."""
import pytest
import torch

from oracle import block

F8 = torch.float64


def randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F8)


def act(z, activation):
    return {None: lambda t: t, "relu": torch.relu, "silu": torch.nn.functional.silu}[activation](z)


@pytest.mark.parametrize("activation", [None, "relu", "silu"])
@pytest.mark.parametrize("shape,groups", [((3, 6), 2), ((2, 5, 12), 4), ((2, 3, 4, 10), 1), ((2, 7, 5), 5)])
def test_group_norm(shape, groups, activation):
    C = shape[-1]
    x, w, b, g = (randn(i, *s).requires_grad_() for i, s in enumerate((shape, (C,), (C,), shape)))
    y = torch.nn.functional.group_norm(x.movedim(-1, 1), groups, w, b, 1e-5).movedim(1, -1)
    y = act(y, activation)
    want = torch.autograd.grad((y * g).sum(), (x, w, b))
    got, mean, rstd, grads, _ = block.group_norm(x, groups, w, b, 1e-5, activation, g=g)
    torch.testing.assert_close(got, y.detach(), rtol=1e-12, atol=1e-12)
    for n, t in zip(("x", "weight", "bias"), want):
        torch.testing.assert_close(grads[n], t, rtol=1e-10, atol=1e-11)
    flat = x.detach().reshape(shape[0], -1, groups, C // groups)
    torch.testing.assert_close(mean, flat.mean((1, 3)))
    torch.testing.assert_close(rstd, (flat.var((1, 3), unbiased=False) + 1e-5).rsqrt())


def test_group_norm_lengths():
    x, w, b, g = randn(1, 4, 9, 6), randn(2, 6), randn(3, 6), randn(4, 4, 9, 6)
    lens = torch.tensor([9, 0, 4, 30], dtype=torch.int32)
    y, mean, rstd, grads, _ = block.group_norm(x, 3, w, b, 1e-5, "silu", lens, g)
    total = torch.zeros(6, dtype=F8)
    for i, n in enumerate((9, 0, 4, 9)):
        assert not y[i, n:].any() and not grads["x"][i, n:].any()
        if n == 0:
            assert not mean[i].any() and not rstd[i].any()
            continue
        wy, wm, wr, wg, _ = block.group_norm(x[i:i + 1, :n], 3, w, b, 1e-5, "silu", None, g[i:i + 1, :n])
        torch.testing.assert_close(y[i, :n], wy[0])
        torch.testing.assert_close(mean[i], wm[0])
        torch.testing.assert_close(grads["x"][i, :n], wg["x"][0])
        total += wg["weight"]
    torch.testing.assert_close(grads["weight"], total)


def plain(x, gate, state, n, blend, reverse):
    """One sequence as autograd sees it."""
    h, ys = state, [None] * n
    for s in range(n):
        t = n - 1 - s if reverse else s
        a = torch.sigmoid(gate[t])
        h = a * h + ((1 - a) * x[t] if blend else x[t])
        ys[t] = h
    return ys, h


@pytest.mark.parametrize("blend", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
def test_gated_recurrence(blend, reverse):
    B, L, C = 4, 70, 3
    x, gate, state, g, g_last = (randn(i, *s) for i, s in enumerate(((B, L, C), (B, L, C), (B, C), (B, L, C), (B, C))))
    lens = torch.tensor([70, 0, 65, 1], dtype=torch.int32)
    got = block.gated_recurrence(x, gate, state, lens, blend, reverse, g, g_last)
    for b, n in enumerate(lens.tolist()):
        v = [t[b].clone().requires_grad_() for t in (x, gate, state)]
        ys, last = plain(*v, n, blend, reverse)
        loss = (last * g_last[b]).sum()
        for t, y in enumerate(ys):
            torch.testing.assert_close(got["y"][b, t], y.detach(), rtol=1e-12, atol=1e-13)
            loss = loss + (y * g[b, t]).sum()
        torch.testing.assert_close(got["last"][b], last.detach())
        want = torch.autograd.grad(loss, v, allow_unused=True)
        for name, t in zip(("gx", "ggate", "gstate"), want):
            t = torch.zeros_like(got[name][b]) if t is None else t
            torch.testing.assert_close(got[name][b], t, rtol=1e-10, atol=1e-12)
        torch.testing.assert_close(got["states"][b, 0], state[b])
        order = list(range(n))[::-1] if reverse else list(range(n))
        torch.testing.assert_close(got["states"][b, 1], got["y"][b, order[63]] if n >= 64 else got["last"][b])


def test_gated_recurrence_differences():
    x, gate, state, g, g_last = (randn(i, *s) for i, s in enumerate(((1, 6, 2), (1, 6, 2), (1, 2), (1, 6, 2), (1, 2))))

    def value(x, gate, state):
        v = block.gated_recurrence(x, gate, state, blend=True)
        return float((v["y"] * g).sum() + (v["last"] * g_last).sum())

    got = block.gated_recurrence(x, gate, state, blend=True, g=g, g_last=g_last)
    args = [x, gate, state]
    step = 1e-5
    for k, name in enumerate(("gx", "ggate", "gstate")):
        flat = got[name].reshape(-1)
        for i in range(flat.numel()):
            v = []
            for sign in (1, -1):
                moved = [t.clone() for t in args]
                moved[k].view(-1)[i] += sign * step
                v.append(value(*moved))
            assert abs((v[0] - v[1]) / (2 * step) - float(flat[i])) < 1e-8


@pytest.mark.parametrize("blend", [False, True])
def test_bounds_hold_for_32_bits(blend):
    """The bounds cover a plain 32-bit evaluation, and are no looser than a
    thousand times its errors."""
    B, L, C = 2, 200, 5
    x, gate, state = randn(1, B, L, C).float(), (randn(2, B, L, C) * 2 + 2).float(), randn(3, B, C).float()
    want = block.gated_recurrence(x, gate, state, blend=blend)
    for b in range(B):
        ys, last = plain(x[b], gate[b], state[b], L, blend, False)
        err = (torch.stack(ys).double() - want["y"][b]).abs()
        assert (err <= want["y_bound"][b]).all()
        assert err.max() * 1000 > want["y_bound"][b].max()
