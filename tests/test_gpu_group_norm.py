"""Group norm with an activation, channels last, and its gradients on the GPU
against plain forms in float64.

Tolerances are bounds of rounding, u = 2^-24.  No value here passes through
more than K = 100 roundings on its way into a group's mean or mean square (a
thread's rows, the row-threads, of which 500 x 3 has 85, and trees over channels
and parts; the cases of test_in_parts say their own), so the mean is off by K u
of the largest |x| of the sample, and

    xh = (x - mean) rstd  by  xe = K u (top rstd + |xh|),
    z = xh w + b          by  ze = |w| xe + 4 u (|z| + |b|),
    silu and its derivative have slopes of at most 1.1 and 0.5, and 12 + |z| roundings.

A parameter's gradient adds up to 256 row-threads and then 64 others in order, W
= 320 in all.

A result in bf16 is rounded once more, by 2^-8 relative.
"""
import pytest
import torch

from deformable_convolution_amd import dc1d, sequence
from oracle import block

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16, F8 = torch.float32, torch.bfloat16, torch.float64
U = 2.0 ** -24
K, W = 100, 320
ACTS = [None, "relu", "silu"]

SHAPES = [
    ((1, 1), 1), ((3, 7), 7), ((16, 512), 8), ((5, 64), 4), ((7, 513), 19), ((70, 24), 3), ((9, 2048), 4), ((3, 4100), 2), ((2, 9000), 1),
    ((2, 5, 1), 1), ((2, 3, 6), 3), ((1, 4, 8), 8), ((2, 33, 64), 1), ((2, 33, 64), 8), ((2, 83, 512), 32), ((1, 1000, 48), 6),
    ((3, 257, 255), 17), ((2, 28, 28, 64), 8), ((2, 7, 9, 30), 5), ((1, 3000, 40), 4), ((2, 300, 1030), 10), ((1, 40, 2056), 8),
    ((1, 3, 5000), 5), ((2, 17, 12), 12), ((300, 2, 16), 2), ((1, 500, 3), 3), ((1, 500, 3), 1), ((4, 784, 96), 32), ((2, 64, 768), 96),
    ((65, 5, 33), 11), ((1, 2000, 129), 3), ((2, 1, 40), 5), ((40, 9, 1), 1), ((1, 1, 17, 264), 33), ((70, 890), 1), ((5, 52, 578), 1), ((3, 200, 99), 3), ((2, 100, 510), 2),
]


def randn(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype).to(DEV)


def inputs(shape, dtype, seed, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    C = shape[-1]
    return (randn(g, *shape, dtype=dtype, scale=1.5, shift=shift), randn(g, C, dtype=dtype, scale=0.3, shift=1.0),
            randn(g, C, dtype=dtype, scale=0.3), randn(g, *shape, dtype=dtype))


def within(got, want, bound, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, what
    bad = ~((got - want).abs() <= bound) & (got != want)
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        bb = bound.expand_as(want)[i] if torch.is_tensor(bound) else bound
        raise AssertionError("%s: %d of %d outside, first at %s: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(bb)))


def once(want, dtype):
    return want.abs() * ((2.0 ** -8 if dtype == BF16 else 4 * U) * 1.01)


def widths(x, w, b, full, lens=None, K=K):
    """xe and ze of every element."""
    v = x.detach().cpu().double()
    if lens is not None:
        see = torch.arange(v.shape[1]).view(1, -1, 1) < lens.cpu().view(-1, 1, 1)
        v = torch.where(see, v, torch.zeros_like(v))
    top = v.abs().amax(tuple(range(1, v.dim())), keepdim=True)
    xe = K * U * (top * full["r"] + full["xh"].abs())
    wa = 1.0 if w is None else w.cpu().double().abs()
    ba = 0.0 if b is None else b.cpu().double().abs()
    return top, xe, wa * xe + 4 * U * (full["z"].abs() + ba)


def check(x, groups, w, b, go, activation, lens=None, eps=1e-5, K=K, W=W):
    dtype = x.dtype
    wy, wm, wr, grads, full = block.group_norm(x, groups, w, b, eps, activation, lens, go)
    top, xe, ze = widths(x, w, b, full, lens, K)
    y, mean, rstd = sequence.group_norm(x, groups, w, b, eps, activation, lens, with_stats=True)
    t = top.reshape(-1, 1)
    within(mean, wm, K * U * t, "mean")
    within(rstd, wr, wr * K * U * (1 + t * wr) ** 2, "rstd")
    slack = (12 + full["z"].abs()) * U
    within(y, wy, 1.1 * ze + slack * wy.abs() + once(wy, dtype), "y")
    got = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, activation, lens)
    ga = go.detach().cpu().double().abs()
    if lens is not None:
        ga = torch.where(full["r"] > 0, ga, torch.zeros_like(ga))
    ge = slack * full["gz"].abs()
    if activation == "silu":
        ge = ge + ga * (0.5 * ze + slack)
    elif activation == "relu":
        ge = ge + ga * (full["z"].abs() <= ze)  # the other side of the step
    wa = 1.0 if w is None else w.cpu().double().abs()
    ue = wa * ge + 2 * U * full["u"].abs()
    n = shape_mean(full["r"], groups)
    xh, u, r = full["xh"].abs(), full["u"].abs(), full["r"]
    e = ue + n(ue) + xh * n(ue * xh + u * xe) + xe * full["aux"] + K * U * (u + full["au"] + xh * full["aux"])
    within(got["x"], grads["x"], r * e * 1.05 + once(grads["x"], dtype), "grad x")
    rest = tuple(range(x.dim() - 1))
    within(got["weight"], grads["weight"], (ge * xh + full["gz"].abs() * xe + W * U * full["gz"].abs() * xh).sum(rest) * 1.05 +
           once(grads["weight"], dtype), "grad weight")
    within(got["bias"], grads["bias"], (ge + W * U * full["gz"].abs()).sum(rest) * 1.05 + once(grads["bias"], dtype), "grad bias")
    return y, mean, rstd, got


def shape_mean(r, groups):
    """The mean over a group's elements that count (r > 0)."""
    B, C = r.shape[0], r.shape[-1]
    n = (r > 0).double().reshape(B, -1, groups, C // groups).sum((1, 3), keepdim=True).clamp(min=1)

    def mean(t):
        v = t.reshape(B, -1, groups, C // groups)
        return (v.sum((1, 3), keepdim=True) / n).expand_as(v).reshape(t.shape)

    return mean


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", SHAPES)
def test_group_norm(shape, groups, dtype):
    print("group norm", shape, groups, dtype, flush=True)
    x, w, b, go = inputs(shape, dtype, 1)
    for activation in ACTS:
        y, mean, rstd, got = check(x, groups, w, b, go, activation)
        assert torch.equal(y, sequence.group_norm(x, groups, w, b, activation=activation))
        again = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, activation)
        assert all(torch.equal(got[n], again[n]) for n in got)
        for n in got:
            alone = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, activation, need=(n,))
            assert list(alone) == [n] and torch.equal(alone[n], got[n])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("given", [(False, False), (True, False), (False, True)])
def test_without_parameters(given, dtype):
    x, w, b, go = inputs((3, 50, 48), dtype, 2)
    for activation in ACTS:
        check(x, 6, w if given[0] else None, b if given[1] else None, go, activation)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("L,C,groups", [(9, 8, 2), (83, 512, 8), (257, 255, 17), (1100, 40, 1), (40, 3, 3), (600, 1030, 10), (30, 2056, 4)])
def test_lengths(L, C, groups, dtype):
    """Lengths of 0 and 1, past the end and below 0; what stands in the padding reaches nothing."""
    print("group norm lengths", L, C, groups, dtype, flush=True)
    x, w, b, go = inputs((6, L, C), dtype, 3)
    lens = torch.tensor([L, 0, 1, L - 3, L + 7, -2], dtype=torch.int32, device=DEV)
    at = torch.arange(L, device=DEV).view(1, L, 1) >= lens.view(-1, 1, 1)
    for activation in ACTS:
        y, mean, rstd, got = check(x, groups, w, b, go, activation, lens)
        for junk in (float("nan"), float("inf")):
            xj, gj = x.masked_fill(at, junk), go.masked_fill(at, -junk)
            yj = sequence.group_norm(xj, groups, w, b, activation=activation, lens=lens)
            assert torch.equal(y, yj)
            again = sequence.group_norm_backward(xj, groups, gj, mean, rstd, w, b, activation, lens)
            assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", [((4, 64), 4), ((2, 300, 48), 6), ((3, 257, 255), 17), ((1, 3000, 264), 1), ((2, 40, 2056), 8), ((3, 70, 198), 2)])
def test_in_place_and_off_alignment(shape, groups, dtype):
    x, w, b, go = inputs(shape, dtype, 4)
    want, mean, rstd = sequence.group_norm(x, groups, w, b, activation="silu", with_stats=True)
    grads = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, "silu")
    same = x.clone()
    assert sequence.group_norm(same, groups, w, b, activation="silu", out=same) is same
    assert torch.equal(same, want)

    def shifted(t, by):
        buf = torch.full((t.numel() + 64,), 7.0, dtype=t.dtype, device=DEV)
        v = buf[by:by + t.numel()].view(t.shape)
        v.copy_(t)
        return buf, v

    for by in (1, 3):
        buf, xs = shifted(x, by)
        _, ws = shifted(w, by)
        _, bs = shifted(b, 2)
        _, gs = shifted(go, by + 1)
        assert torch.equal(sequence.group_norm(xs, groups, ws, bs, activation="silu"), want)
        obuf, ys = shifted(torch.zeros_like(x), by + 1)
        sequence.group_norm(xs, groups, ws, bs, activation="silu", out=ys)
        assert torch.equal(ys, want)
        assert (obuf[:by + 1] == 7).all() and (obuf[by + 1 + x.numel():] == 7).all()  # nothing around it is written
        again = sequence.group_norm_backward(xs, groups, gs, mean, rstd, ws, bs, "silu")
        assert all(torch.equal(again[n], grads[n]) for n in grads)


# Samples too large to hold: with fewer parts' statistics than every workgroup joins itself and with more, channels in
# several tiles, parts whose second pass is split, one and few channels.  K: 8 rows of a thread, the row-threads (253 of
# 8 channels), then a part's channels and the parts over 64 lanes or more (5000 channels: 79 of a lane).
PARTS = [((2, 5000, 64), 1, 100), ((2, 3000, 264), 3, 100), ((3, 1300, 512), 512, 192), ((2, 6000, 96), 96, 100),
         ((1, 4100, 1030), 2, 100), ((1, 300, 5000), 1, 120), ((1, 2000, 2056), 1, 100), ((2, 700, 4104), 54, 100), ((1, 600, 4096), 512, 100), ((1, 30000, 8), 1, 320)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups,k", PARTS)
def test_in_parts(shape, groups, k, dtype):
    print("group norm in parts", shape, groups, dtype, flush=True)
    x, w, b, go = inputs(shape, dtype, 10)
    y, mean, rstd, got = check(x, groups, w, b, go, "silu", K=k, W=max(k, W))
    assert torch.equal(y, sequence.group_norm(x, groups, w, b, activation="silu"))
    same = x.clone()
    sequence.group_norm(same, groups, w, b, activation="silu", out=same)
    assert torch.equal(same, y)
    over = go.clone()
    again = sequence.group_norm_backward(x, groups, over, mean, rstd, w, b, "silu")
    assert all(torch.equal(got[n], again[n]) for n in got)
    # lengths that end inside a part, at its first position and ahead of it
    L = shape[1]
    lens = torch.tensor([L - 7, 9, 1][:shape[0]], dtype=torch.int32, device=DEV)
    check(x, groups, w, b, go, None, lens, K=k, W=max(k, W))
    # a NaN stays in its group
    plain = sequence.group_norm(x, groups)
    x[0, L // 2, 3] = float("nan")
    y, D, g = sequence.group_norm(x, groups), shape[2] // groups, 3 * groups // shape[2]
    assert y[0, :, g * D:(g + 1) * D].isnan().all()
    y[0, :, g * D:(g + 1) * D] = plain[0, :, g * D:(g + 1) * D]
    assert torch.equal(y, plain)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_samples_in_parts(dtype):
    """Workgroups enough without parts: a second pass of several workgroups to a sample."""
    x, w, b, go = inputs((520, 601, 36), dtype, 11)
    lens = torch.full((520,), 601, dtype=torch.int32, device=DEV)
    lens[::3], lens[1::5], lens[7] = 300, 2, 0
    check(x, 1, w, b, go, "relu")
    check(x, 1, w, b, go, "silu", lens)


def test_workspace():
    """A caller's workspace: too small, unaligned and overlapping ones are refused, and what it holds does not matter."""
    x, w, b, go = inputs((2, 5000, 64), F32, 12)
    want = sequence.group_norm(x, 4, w, b, with_stats=True)
    ws = torch.full((1 << 22,), 255, dtype=torch.uint8, device=DEV)
    got = sequence.group_norm(x, 4, w, b, with_stats=True, workspace=ws)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    grads = sequence.group_norm_backward(x, 4, go, want[1], want[2], w, b)
    again = sequence.group_norm_backward(x, 4, go, want[1], want[2], w, b, workspace=ws.fill_(127))
    assert all(torch.equal(grads[n], again[n]) for n in grads)
    for bad in (ws[:128], ws[8:]):
        with pytest.raises(dc1d.Dc1dValueError):
            sequence.group_norm(x, 4, w, b, workspace=bad)
        with pytest.raises(dc1d.Dc1dValueError):
            sequence.group_norm_backward(x, 4, go, want[1], want[2], w, b, workspace=bad)
    inside = x.view(-1).view(torch.uint8)[:1 << 20]
    with pytest.raises(dc1d.Dc1dValueError):
        sequence.group_norm(x, 4, w, b, workspace=inside)


@pytest.mark.parametrize("shape", [((1 << 20) + 3, 2100), (1, (1 << 20) + 3, 2100)])
def test_past_32_bits(shape):
    """4.4 GB: many samples of one position, and one of many.  The last rows and the statistics; K = 1400: 1366 rows of
    a thread, 8 to a batch that is joined in 3 roundings, then 256 parts."""
    C, rows = shape[-1], (1 << 20) + 3
    x = torch.empty(shape, dtype=BF16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(13)
    flat = x.view(rows, C)
    for i in range(0, rows, 1 << 17):
        part = flat[i:i + (1 << 17)]
        part.copy_(torch.randn(part.shape, generator=gen, device=DEV, dtype=F32) + 1)
    tail = flat[-5:].cpu().double()
    k, groups = 1400, 3
    if len(shape) == 2:
        m = tail.view(5, groups, -1).mean(2)
        var = ((tail.view(5, groups, -1) - m[..., None]) ** 2).mean(2)
    else:
        v = [flat[i:i + (1 << 17)].double().view(-1, groups, C // groups) for i in range(0, rows, 1 << 17)]
        n = rows * (C // groups)
        m = sum(t.sum((0, 2)) for t in v) / n
        var = (sum(((t - m[None, :, None]) ** 2).sum((0, 2)) for t in v) / n).cpu().expand(5, groups)
        m = m.cpu().expand(5, groups)
        del v
    r = (var + 1e-5) ** -0.5
    y, mean, rstd = sequence.group_norm(x, groups, out=x, with_stats=True)
    last = 5 if len(shape) == 2 else 1
    top = 8.0  # |x| below, of 2^31 normal numbers about 1
    within(mean[-last:], m[-last:], k * U * top, "mean")
    within(rstd[-last:], r[-last:], k * U * (1 + top) ** 2, "rstd")
    want = ((tail.view(5, groups, -1) - m[..., None]) * r[..., None]).view(5, C)
    within(y.view(rows, C)[-5:], want, k * U * 2 * top + once(want, BF16), "y")


def test_large_mean():
    """The variance is that of centred values: a mean of 1000 deviations costs the digits of the mean alone,
    also behind a run of zeros."""
    g = torch.Generator().manual_seed(5)
    for shape, groups in (((2, 4000, 32), 2), ((2, 60, 32), 2), ((50, 512), 4)):
        x = randn(g, *shape, shift=1000.0)
        if len(shape) == 3:
            x[1, :shape[1] // 10] = 0.0
        check(x, groups, None, None, randn(g, *shape), None)


def test_equal_values_and_eps():
    x = torch.full((2, 30, 16), 3.0, device=DEV)
    y, mean, rstd = sequence.group_norm(x, 4, with_stats=True)
    assert not y.any() and (mean == 3.0).all() and ((rstd - 1e-5 ** -0.5).abs() <= 4 * U * 317).all()
    x, w, b, go = inputs((2, 30, 16), F32, 6)
    for eps in (0.0, 1e-3, 10.0):
        check(x, 4, w, b, go, "silu", eps=eps)


def test_nan_stays_in_its_group():
    x, w, b, go = inputs((3, 40, 32), F32, 7)
    want = sequence.group_norm(x, 4, w, b, activation="relu")
    x[1, 7, 9] = float("nan")
    y = sequence.group_norm(x, 4, w, b, activation="relu")
    assert y[1, :, 8:16].isnan().all()
    y[1, :, 8:16] = want[1, :, 8:16]
    assert torch.equal(y, want)


def test_empty():
    for shape in ((0, 8), (0, 5, 8), (3, 0, 8)):
        x = torch.zeros(shape, device=DEV)
        y, mean, rstd = sequence.group_norm(x, 2, with_stats=True)
        assert y.shape == x.shape and mean.shape == (shape[0], 2) and not mean.any() and not rstd.any()
        got = sequence.group_norm_backward(x, 2, x, mean, rstd)
        assert got["x"].shape == x.shape and not got["weight"].any() and not got["bias"].any()
        assert got["weight"].shape == (8,)


def test_gradient_against_differences():
    """A directional derivative in float32 sums: the difference quotient of steps of 2^-7 is off by its
    curvature (h^2 / 6 of a third derivative, bounded here by 100 of the gradient's size) and by the sums'
    rounding, 2^-18 of the absolute sum over the step."""
    x, w, b, go = inputs((2, 20, 16), F32, 8)
    _, mean, rstd = sequence.group_norm(x, 4, w, b, activation="silu", with_stats=True)
    got = sequence.group_norm_backward(x, 4, go, mean, rstd, w, b, "silu")
    for n, t in (("x", x), ("weight", w), ("bias", b)):
        d = randn(torch.Generator().manual_seed(9), *t.shape)
        d = d / d.norm()
        h = 2.0 ** -7
        v = []
        for sign in (1, -1):
            args = {"x": x, "weight": w, "bias": b}
            args[n] = t + sign * h * d
            v.append((sequence.group_norm(args["x"], 4, args["weight"], args["bias"], activation="silu").double() * go.double()).sum())
        slope = float((v[0] - v[1]) / (2 * h))
        size = float(got[n].double().norm())
        assert abs(slope - float((got[n].double() * d.double()).sum())) <= size * (100 * h * h / 6) + 2.0 ** -18 * float(
            go.abs().sum()) / h * 2.0 ** -4
