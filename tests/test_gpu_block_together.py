"""The operators of a recurrent block as they are used together: group norm,
the gated recurrence over what it gives, a norm of every position's heads, a
projection from attention's side of the package left out.  Every stage is
checked against its plain form on what the stage before it gave (the
tolerances of the operators' own tests), the whole for its gradients against
differences, and a sequence taken position by position against the whole."""
import pytest
import torch

from deformable_convolution_amd import sequence
from oracle import block
from test_gpu_gated_recurrence import within as within_recurrence
from test_gpu_group_norm import check as check_norm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


class Block:
    """x -> silu(norm(x)) = h; the recurrence of h under the gates -> s; norm over each position's heads -> y."""

    def __init__(self, C, groups, heads, dtype, seed, blend=True):
        g = torch.Generator().manual_seed(seed)
        rand = lambda shift: (0.3 * torch.randn(C, generator=g) + shift).to(dtype).to(DEV)  # noqa: E731
        self.w, self.b, self.hw, self.hb = rand(1.0), rand(0.0), rand(1.0), rand(0.0)
        self.groups, self.heads, self.C, self.blend = groups, heads, C, blend

    def forward(self, x, gate, state=None, lens=None):
        h, mean, rstd = sequence.group_norm(x, self.groups, self.w, self.b, activation="silu", lens=lens, with_stats=True)
        s, last, states = sequence.gated_recurrence(h, gate, state, lens, self.blend, with_states=True)
        y, hmean, hrstd = sequence.group_norm(s.reshape(-1, self.C), self.heads, self.hw, self.hb, with_stats=True)
        return y.view_as(x), last, (x, gate, h, mean, rstd, s, states, hmean, hrstd, lens)

    def backward(self, kept, gy, g_last):
        x, gate, h, mean, rstd, s, states, hmean, hrstd, lens = kept
        top = sequence.group_norm_backward(s.reshape(-1, self.C), self.heads, gy.reshape(-1, self.C), hmean, hrstd, self.hw, self.hb)
        gs = top["x"].view_as(s)
        mid = sequence.gated_recurrence_backward(h, gate, states, gs, g_last, lens, self.blend, grads={"x": gs})
        low = sequence.group_norm_backward(x, self.groups, mid["x"], mean, rstd, self.w, self.b, "silu", lens)
        return {"x": low["x"], "gate": mid["gate"], "state": mid["state"], "w": low["weight"], "b": low["bias"],
                "hw": top["weight"], "hb": top["bias"]}


def inputs(B, L, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g).to(DEV)  # noqa: E731
    return (rand(B, L, C).to(dtype), (2 * rand(B, L, C) + 1).to(dtype), rand(B, C), rand(B, L, C).to(dtype), rand(B, C))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups,heads", [((2, 83, 64), 8, 4), ((1, 700, 40), 5, 1), ((3, 130, 48), 1, 48)])
def test_stage_by_stage(shape, groups, heads, dtype):
    blk = Block(shape[2], groups, heads, dtype, 1)
    x, gate, state, gy, g_last = inputs(*shape, dtype, 2)
    lens = torch.tensor([shape[1], 40, 0][:shape[0]], dtype=torch.int32, device=DEV)
    y, last, kept = blk.forward(x, gate, state, lens)
    h, s, states = kept[2], kept[5], kept[6]
    grads = blk.backward(kept, gy, g_last)
    h1, _, _, _ = check_norm(x, groups, blk.w, blk.b, gy, "silu", lens)
    assert torch.equal(h1, h)
    top = check_norm(s.reshape(-1, shape[2]), heads, blk.hw, blk.hb, gy.reshape(-1, shape[2]), None)
    assert torch.equal(top[0].view_as(y), y) and torch.equal(top[3]["weight"], grads["hw"])
    gs = top[3]["x"].view_as(s)
    want = block.gated_recurrence(h, gate, state, lens, True, False, gs, g_last)
    for name, t, dt in (("y", s, dtype), ("last", last, F32), ("states", states, F32), ("ggate", grads["gate"], dtype),
                        ("gstate", grads["state"], F32)):
        within_recurrence(t, want, name, dt, "block")
    mid = sequence.gated_recurrence_backward(h, gate, states, gs, g_last, lens, True)
    low = check_norm(x, groups, blk.w, blk.b, mid["x"], "silu", lens)[3]
    assert torch.equal(low["x"], grads["x"]) and torch.equal(low["weight"], grads["w"]) and torch.equal(low["bias"], grads["b"])


def test_gradients_against_differences():
    """Directional derivatives: the quotient of steps of 2^-7 is off by its curvature (h^2 / 6 of a third derivative,
    bounded here by 100 of the gradient's size) and by rounding, 2^-20 of the absolute sum over the step (three
    stages, each as in the operators' own tests)."""
    blk = Block(24, 3, 4, F32, 3)
    x, gate, state, gy, g_last = inputs(2, 70, 24, F32, 4)
    _, _, kept = blk.forward(x, gate, state)
    got = blk.backward(kept, gy, g_last)
    at = {"x": x, "gate": gate, "state": state, "w": blk.w, "b": blk.b, "hw": blk.hw, "hb": blk.hb}
    gen = torch.Generator().manual_seed(5)
    for n, t in at.items():
        d = torch.randn(t.shape, generator=gen).to(DEV)
        d = d / d.norm()
        h, v, size = 2.0 ** -7, [], 0.0
        for sign in (1, -1):
            args = dict(at)
            args[n] = t + sign * h * d
            blk.w, blk.b, blk.hw, blk.hb = (args[k] for k in ("w", "b", "hw", "hb"))
            y, last, _ = blk.forward(args["x"], args["gate"], args["state"])
            v.append((y.double() * gy.double()).sum() + (last.double() * g_last.double()).sum())
            size = float((y * gy).abs().sum()) + float((last * g_last).abs().sum())
        blk.w, blk.b, blk.hw, blk.hb = (at[k] for k in ("w", "b", "hw", "hb"))
        slope = float((v[0] - v[1]) / (2 * h))
        assert abs(slope - float((got[n].double() * d.double()).sum())) <= float(got[n].double().norm()) * 100 * h * h / 6 + (
            2.0 ** -20 * size / h), n


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_position_by_position(dtype):
    """Norms of single positions and the state carried from call to call give what a whole sequence gives, up to
    the roundings of its plain form; here the first norm too is one of each position."""
    B, L, C = 3, 70, 48
    blk = Block(C, 6, 4, dtype, 6)
    x, gate, state, _, _ = inputs(B, L, C, dtype, 7)
    whole = sequence.group_norm(x.reshape(-1, C), 6, blk.w, blk.b, activation="silu").view_as(x)
    steps = torch.stack([sequence.group_norm(x[:, t].contiguous(), 6, blk.w, blk.b, activation="silu") for t in range(L)], 1)
    check_norm(x.reshape(-1, C), 6, blk.w, blk.b, x.reshape(-1, C), "silu")
    check_norm(x[:, 5].contiguous(), 6, blk.w, blk.b, x[:, 6].contiguous(), "silu")
    want = block.gated_recurrence(steps, gate, state, None, True)
    s = state.clone()
    ys = [sequence.gated_recurrence(steps[:, t:t + 1], gate[:, t:t + 1], s, blend=True, last=s)[0] for t in range(L)]
    within_recurrence(torch.cat(ys, 1), want, "y", dtype, "steps")
    within_recurrence(s, want, "last", F32, "steps")
    y, last = sequence.gated_recurrence(steps, gate, state, blend=True)
    within_recurrence(y, want, "y", dtype, "whole")
    within_recurrence(last, want, "last", F32, "whole")
    assert (whole - steps).abs().max() <= whole.abs().max() * torch.finfo(dtype).eps
