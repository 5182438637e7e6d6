"""The gated linear recurrence and its gradients on the GPU against a plain form
in float64, which also gives the bounds (oracle/block.py: errors of 32-bit
arithmetic carried along the sequence); a result in bf16 is rounded once more,
by 2^-8 relative.  The relative bounds hold for normal numbers: what lies below
the least of them, 2^-126, or is a product of one that does and of factors below
1, is off by less than 2^-126 if it becomes 0."""
import pytest
import torch

from deformable_convolution_amd import dc1d, sequence
from oracle import block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16

SHAPES = [(1, 1, 1), (2, 1, 5), (16, 1, 512), (3, 2, 4), (1, 2, 2), (2, 4, 9), (2, 63, 8), (2, 64, 7), (1, 65, 33), (2, 130, 64),
          (1, 700, 20), (3, 129, 130), (2, 300, 3), (2, 83, 96), (1, 1500, 5), (70, 70, 6), (1, 257, 300), (2, 3, 515)]


def randn(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def inputs(B, L, C, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (randn(g, B, L, C, dtype=dtype), randn(g, B, L, C, dtype=dtype, scale=2.0, shift=2.0), randn(g, B, C),
            randn(g, B, L, C, dtype=dtype), randn(g, B, C))


def within(got, want, name, dtype, what):
    w, bound = want[name], want[name + "_bound"]
    assert got.shape == w.shape and got.dtype == dtype, (what, got.shape, got.dtype)
    got = got.cpu().double()
    bound = bound + w.abs() * ((2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * 1.01) + 2.0 ** -126
    bad = ~((got - w).abs() <= bound) & (got != w)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s %s: %d of %d outside, first at %s: got %r, want %r, bound %r" % (
            what, name, int(bad.sum()), bad.numel(), i, float(got[i]), float(w[i]), float(bound[i])))


def check(x, gate, state, go, g_last, lens=None, blend=False, reverse=False, what=""):
    dtype = x.dtype
    want = block.gated_recurrence(x, gate, state, lens, blend, reverse, go, g_last)
    y, last, states = sequence.gated_recurrence(x, gate, state, lens, blend, reverse, with_states=True)
    for name, t, dt in (("y", y, dtype), ("last", last, F32), ("states", states, F32)):
        within(t, want, name, dt, what)
    got = sequence.gated_recurrence_backward(x, gate, states, go, g_last, lens, blend, reverse)
    for name, key, dt in (("gx", "x", dtype), ("ggate", "gate", dtype), ("gstate", "state", F32)):
        within(got[key], want, name, dt, what)
    return y, last, states, got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated_recurrence(shape, dtype):
    print("gated recurrence", shape, dtype, flush=True)
    x, gate, state, go, g_last = inputs(*shape, dtype, 1)
    for blend, reverse in ((False, False), (True, False), (False, True), (True, True)):
        y, last, states, got = check(x, gate, state, go, g_last, None, blend, reverse, "blend %d reverse %d" % (blend, reverse))
        y2, last2 = sequence.gated_recurrence(x, gate, state, blend=blend, reverse=reverse)
        assert torch.equal(y, y2) and torch.equal(last, last2)
        again = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=blend, reverse=reverse)
        assert all(torch.equal(got[n], again[n]) for n in got)
        for n in got:
            alone = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=blend, reverse=reverse, need=(n,))
            assert list(alone) == [n] and torch.equal(alone[n], got[n])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(520, 140, 5), (1, 140, 33001), (1, 40000, 4), (2, 9000, 70), (2, 1400, 3), (5, 700, 2049)])
def test_many_chains_and_many_segments(shape, dtype):
    """Sequences and channels enough for one pass over several tiles; long ones cut into many segments."""
    print("gated recurrence", shape, dtype, flush=True)
    x, gate, state, go, g_last = inputs(*shape, dtype, 11)
    lens = torch.full((shape[0],), shape[1], dtype=torch.int32, device=DEV)
    lens[-1] = shape[1] - 67
    check(x, gate, state, go, g_last, None, False, True)
    check(x, gate, state, go, g_last, lens, True, False)


@pytest.mark.parametrize("reverse", [False, True])
def test_rows_far_apart(reverse):
    """Rows 33 MB apart, which a tile's 32-bit offsets do not span, and beside them rows that are."""
    B, L, C = 1, 4, 8
    x, gate, state, go, g_last = inputs(B, L, C, F32, 12)
    step = (1 << 23) + 5
    far = []
    for t in (x, gate, go):
        v = torch.zeros(step * L, device=DEV).as_strided((B, L, C), (step * L, step, 1))
        v.copy_(t)
        far.append(v)
    check(far[0], far[1], state, far[2], g_last, None, True, reverse)
    check(far[0], gate, state, go, g_last, None, False, reverse)
    check(x, gate, state, far[2], g_last, None, False, reverse)
    y = torch.zeros(step * L, device=DEV).as_strided((B, L, C), (step * L, step, 1))
    sequence.gated_recurrence(x, gate, state, blend=True, reverse=reverse, out=y)
    want = block.gated_recurrence(x, gate, state, None, True, reverse)
    within(y, want, "y", F32, "far output")


def test_past_32_bits():
    """4.4 GB a tensor; a gate of -infinity 150 positions ahead of the end, from which the plain form starts."""
    L, C, tail = (1 << 20) + 77, 2100, 150
    x = torch.empty((1, L, C), dtype=BF16, device=DEV)
    gate = torch.empty((1, L, C), dtype=BF16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(14)
    for i in range(0, L, 1 << 17):
        for t, up in ((x, 0.0), (gate, 2.0)):
            part = t[0, i:i + (1 << 17)]
            part.copy_(torch.randn(part.shape, generator=gen, device=DEV, dtype=F32) + up)
    gate[:, L - tail] = -float("inf")
    ends = [t[:, L - tail:].clone() for t in (x, gate)]
    go = ends[0].flip(1).contiguous()
    want = block.gated_recurrence(ends[0], ends[1], None, None, False, False, go, None)
    wide = torch.zeros_like(x)
    wide[:, L - tail:] = go
    y, last, states = sequence.gated_recurrence(x, gate, with_states=True)
    within(y[:, L - tail:], want, "y", BF16, "tail")
    within(last, want, "last", F32, "tail")
    del y
    got = sequence.gated_recurrence_backward(x, gate, states, wide, grads={"x": wide})
    within(got["x"][:, L - tail:], want, "gx", BF16, "tail")
    # the state ahead of the tail is another one than the plain form's, and its gate lets none of it through
    within(got["gate"][:, L - tail:], want, "ggate", BF16, "tail")
    assert not got["x"][:, :L - tail].any() and not got["gate"][:, :L - tail].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_without_states(dtype):
    x, gate, _, go, _ = inputs(2, 90, 12, dtype, 2)
    check(x, gate, None, go, None)
    check(x, gate, None, go, None, blend=True, reverse=True)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,C", [(5, 8), (64, 33), (129, 3), (200, 70), (1300, 4)])
def test_lengths(L, C, dtype):
    """Lengths of 0 and 1, past the end and below 0, around the kept states; what stands in the padding reaches nothing."""
    print("gated recurrence lengths", L, C, dtype, flush=True)
    n = [L, 0, 1, L - 1, L + 5, -3, min(L, 63), min(L, 65)]
    x, gate, state, go, g_last = inputs(len(n), L, C, dtype, 3)
    lens = torch.tensor(n, dtype=torch.int32, device=DEV)
    at = torch.arange(L, device=DEV).view(1, L, 1) >= lens.view(-1, 1, 1)
    for blend, reverse in ((False, False), (True, True)):
        y, last, states, got = check(x, gate, state, go, g_last, lens, blend, reverse)
        assert not y[at.expand_as(y)].any() and torch.equal(last[1], state[1]) and torch.equal(got["state"][1], g_last[1])
        for junk in (float("nan"), float("inf")):
            args = [t.masked_fill(at, junk) for t in (x, gate, go)]
            again = sequence.gated_recurrence(args[0], args[1], state, lens, blend, reverse, with_states=True)
            assert all(torch.equal(p, q) for p, q in zip(again, (y, last, states)))
            g2 = sequence.gated_recurrence_backward(args[0], args[1], states, args[2], g_last, lens, blend, reverse)
            assert all(torch.equal(got[k], g2[k]) for k in got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,L,C", [(2, 83, 24), (1, 900, 10), (3, 1, 40)])
def test_layouts(B, L, C, dtype):
    """Slices of one projection, results into slices of one buffer, broadcast gates, results in place, odd alignment."""
    x, gate, state, go, g_last = inputs(B, L, C, dtype, 4)
    y, last, states = sequence.gated_recurrence(x, gate, state, blend=True, with_states=True)
    got = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=True)
    for pad in (0, 1, 3):
        both = torch.full((B, L, 2 * C + pad), 7.0, dtype=dtype, device=DEV)
        xs, gs = both[..., pad:pad + C], both[..., pad + C:]
        xs.copy_(x)
        gs.copy_(gate)
        out = torch.full((B, L, 2 * C + pad), 7.0, dtype=dtype, device=DEV)
        y2, last2 = sequence.gated_recurrence(xs, gs, state, blend=True, out=out[..., pad:pad + C])
        assert torch.equal(y2, y) and torch.equal(last2, last)
        assert (out[..., :pad] == 7).all() and (out[..., pad + C:] == 7).all()
        out.fill_(7.0)
        g2 = sequence.gated_recurrence_backward(xs, gs, states, go, g_last, blend=True,
                                                grads={"x": out[..., pad:pad + C], "gate": out[..., pad + C:]})
        assert all(torch.equal(got[k], g2[k]) for k in got) and (out[..., :pad] == 7).all()
        assert torch.equal(out[..., pad + C:], got["gate"])
        # the results over x, and over grad_out
        y3, _ = sequence.gated_recurrence(xs, gs, state, blend=True, out=xs)
        assert y3.data_ptr() == xs.data_ptr() and torch.equal(y3, y) and torch.equal(gs, gate)
    # batch and position exchanged in memory
    t = [v.transpose(0, 1).clone(memory_format=torch.contiguous_format).transpose(0, 1) for v in (x, gate, go)]  # a clone: go is written below
    assert torch.equal(sequence.gated_recurrence(t[0], t[1], state, blend=True)[0], y)
    g2 = sequence.gated_recurrence_backward(t[0], t[1], states, t[2], g_last, blend=True, grads={"x": t[2]})
    assert all(torch.equal(got[k], g2[k]) for k in got)
    # one gate for all batches, and for all positions
    for shape in ((1, L, C), (B, 1, C), (1, 1, C)):
        small = gate[:shape[0], :shape[1]].clone()
        wide = small.expand(B, L, C)
        check(x, wide, state, go, g_last, None, False, False, "expanded")
    # the state in place, and its gradient over the last one's
    s = state.clone()
    _, back = sequence.gated_recurrence(x, gate, s, blend=True, last=s)
    assert back is s and torch.equal(s, last)
    gl = g_last.clone()
    g2 = sequence.gated_recurrence_backward(x, gate, states, go, gl, blend=True, grads={"state": gl})
    assert torch.equal(gl, got["state"]) and torch.equal(g2["x"], got["x"])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("C", [65, 67, 130, 515])
def test_states_in_place_beside_another_workgroup(C, dtype):
    """A row's last channels are read by the workgroup of its last piece and by the one before it, which may have
    replaced their state by then: y and the gradients are those of states of their own."""
    for B, L in ((40, 1), (3000, 1), (3000, 3), (30, 70)):
        x, gate, state, go, g_last = inputs(B, L, C, dtype, 15)
        want, last, states = sequence.gated_recurrence(x, gate, state, blend=True, with_states=True)
        grads = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=True)
        for _ in range(5):
            s = state.clone()
            y, _ = sequence.gated_recurrence(x, gate, s, blend=True, last=s)
            assert torch.equal(y, want) and torch.equal(s, last)
            gl = g_last.clone()
            got = sequence.gated_recurrence_backward(x, gate, states, go, gl, blend=True, grads={"state": gl})
            assert all(torch.equal(got[n], grads[n]) for n in grads)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_position_by_position(dtype):
    """A sequence taken up again at every position, or in pieces, gives what it gives at once, up to rounding."""
    x, gate, state, go, g_last = inputs(3, 75, 20, dtype, 5)
    want = block.gated_recurrence(x, gate, state)
    s = state.clone()
    ys = [sequence.gated_recurrence(x[:, t:t + 1], gate[:, t:t + 1], s, last=s)[0] for t in range(75)]
    within(torch.cat(ys, 1), want, "y", dtype, "steps")
    within(s, want, "last", F32, "steps")
    s = state.clone()
    ys = [sequence.gated_recurrence(x[:, a:b], gate[:, a:b], s, last=s)[0] for a, b in ((0, 31), (31, 32), (32, 75))]
    within(torch.cat(ys, 1), want, "y", dtype, "pieces")
    within(s, want, "last", F32, "pieces")


@pytest.mark.parametrize("blend", [False, True])
def test_infinite_gates(blend):
    """-infinity starts anew, exactly; +infinity holds the state (exactly from the call's start on; a state that
    was reached inside the call is formed again for each few positions, by other sums of the same terms, whose
    roundings check() bounds)."""
    x, gate, state, go, g_last = inputs(2, 100, 8, F32, 6)
    gate[0, 40] = -float("inf")
    gate[1, 10:90] = float("inf")
    gate[0, 70] = -3.4e38
    gate[1, 95] = 3.4e38
    y, last, states, got = check(x, gate, state, go, g_last, None, blend, False)
    assert torch.equal(y[0, 40], x[0, 40]) and torch.equal(y[0, 70], x[0, 70])
    if blend:
        held, last = sequence.gated_recurrence(x, torch.full_like(gate, float("inf")), state, blend=True)
        assert torch.equal(held, state.unsqueeze(1).expand_as(held)) and torch.equal(last, state)
        assert not got["x"][1, 10:90].any()
    assert not got["gate"][0, 40].any() and not got["gate"][1, 10:90].any()
    # what came before the new start reaches nothing after it
    other = x.clone()
    other[0, :40] = 1e30
    assert torch.equal(sequence.gated_recurrence(other, gate, state, blend=blend)[0][0, 40:], y[0, 40:])


def test_nan_reaches_later_positions_of_its_channel_only():
    x, gate, state, _, _ = inputs(2, 150, 12, F32, 7)
    want, _ = sequence.gated_recurrence(x, gate, state)
    x[1, 77, 5] = float("nan")
    y, last = sequence.gated_recurrence(x, gate, state)
    assert y[1, 77:, 5].isnan().all() and last[1, 5].isnan()
    y[1, 77:, 5] = want[1, 77:, 5]
    assert torch.equal(y, want)


def test_nan_in_gates_and_gradients():
    """A NaN gate reaches its channel's later states and the gradients of it and of the earlier positions, and a
    NaN gradient those of its position and the earlier ones; nothing else, over several segments."""
    x, gate, state, go, g_last = inputs(2, 1500, 12, F32, 13)
    y0, last0, states = sequence.gated_recurrence(x, gate, state, blend=True, with_states=True)
    want = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=True)
    bad = gate.clone()
    bad[1, 777, 5] = float("nan")
    y, last, states2 = sequence.gated_recurrence(x, bad, state, blend=True, with_states=True)
    assert y[1, 777:, 5].isnan().all() and last[1, 5].isnan()
    y[1, 777:, 5] = y0[1, 777:, 5]
    assert torch.equal(y, y0)
    bad = go.clone()
    bad[0, 900, 3] = float("nan")
    got = sequence.gated_recurrence_backward(x, gate, states, bad, g_last, blend=True)
    for n in ("x", "gate"):
        assert got[n][0, :901, 3].isnan().all()
        got[n][0, :901, 3] = want[n][0, :901, 3]
        assert torch.equal(got[n], want[n])
    assert got["state"][0, 3].isnan()
    got["state"][0, 3] = want["state"][0, 3]
    assert torch.equal(got["state"], want["state"])


def test_empty():
    state = torch.randn(3, 8, device=DEV)
    x = torch.zeros(3, 0, 8, device=DEV)
    y, last, states = sequence.gated_recurrence(x, x, state, with_states=True)
    assert y.shape == (3, 0, 8) and torch.equal(last, state) and states.shape == (3, 0, 8)
    got = sequence.gated_recurrence_backward(x, x, states, x, state)
    assert torch.equal(got["state"], state) and got["gate"].shape == (3, 0, 8)
    x = torch.zeros(0, 5, 8, device=DEV)
    y, last, states = sequence.gated_recurrence(x, x, with_states=True)
    assert last.shape == (0, 8) and states.shape == (0, 1, 8)
    assert sequence.gated_recurrence_backward(x, x, states, x)["x"].shape == (0, 5, 8)


def test_workspace():
    """A caller's workspace: too small, unaligned and overlapping ones are refused, and what it holds does not matter."""
    x, gate, state, go, g_last = inputs(1, 2000, 40, F32, 8)
    want = sequence.gated_recurrence(x, gate, state, with_states=True)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    got = sequence.gated_recurrence(x, gate, state, with_states=True, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    for bad in (ws[:256], ws[8:]):
        with pytest.raises(dc1d.Dc1dValueError):
            sequence.gated_recurrence(x, gate, state, workspace=bad)
    grads = sequence.gated_recurrence_backward(x, gate, want[2], go, g_last)
    again = sequence.gated_recurrence_backward(x, gate, want[2], go, g_last, workspace=ws.fill_(127))
    assert all(torch.equal(grads[k], again[k]) for k in grads)


def test_gradient_against_differences():
    """Directional derivatives: the quotient of steps of 2^-7 is off by the curvature (h^2 / 6 of a third
    derivative, bounded here by 100 of the gradient's size) and by rounding, 2^-22 of the absolute sum over the
    step."""
    x, gate, state, go, g_last = inputs(2, 70, 6, F32, 9)
    for blend, reverse in ((False, False), (True, True)):
        _, _, states = sequence.gated_recurrence(x, gate, state, blend=blend, reverse=reverse, with_states=True)
        got = sequence.gated_recurrence_backward(x, gate, states, go, g_last, blend=blend, reverse=reverse)
        for n, t in (("x", x), ("gate", gate), ("state", state)):
            d = randn(torch.Generator().manual_seed(10), *t.shape)
            d = d / d.norm()
            h, v, size = 2.0 ** -7, [], 0.0
            for sign in (1, -1):
                args = {"x": x, "gate": gate, "state": state}
                args[n] = t + sign * h * d
                y, last = sequence.gated_recurrence(args["x"], args["gate"], args["state"], blend=blend, reverse=reverse)
                v.append((y.double() * go.double()).sum() + (last.double() * g_last.double()).sum())
                size = float((y * go).abs().sum())
            slope = float((v[0] - v[1]) / (2 * h))
            assert abs(slope - float((got[n].double() * d.double()).sum())) <= float(got[n].double().norm()) * 100 * h * h / 6 + (
                2.0 ** -22 * size / h)
