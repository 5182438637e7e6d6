"""The sequence operators on the GPU (layer norm, rotary positions, attention
and their gradients) against plain forms in float64, at the sizes, layouts
and masks where such kernels go wrong.

Tolerances are bounds of rounding: unit roundoff u (2^-24 for fp32, 2^-8 for
one rounding to bf16) times the absolute sums of what is added up (see
oracle/sequence.py), with the factors stated at each check.
"""
import math

import pytest
import torch

from deformable_convolution_amd import dc1d, sequence
from oracle import sequence as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U32 = 2.0 ** -24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale + shift).to(dtype)


def within(got, want, bound, what):
    assert got.shape == want.shape, what
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    same = got == want  # infinities
    bad &= ~same
    if bad.any():
        i = tuple(int(v) for v in bad.nonzero()[0])
        bb = bound if not torch.is_tensor(bound) else bound.expand_as(want)[i]
        raise AssertionError("%s: %d of %d outside, first at %s: got %r, want %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got[i]), float(want[i]), float(bb)))


# ---- layer norm ------------------------------------------------------------------

LN_SHAPES = [
    (1, 1), (3, 7), (1, 8), (5, 64), (16, 512), (7, 513), (33, 1024), (2, 2000), (9, 4096), (4, 8192), (3, 8200), (2, 20001),
    (2, 5, 1), (1, 4, 1), (2, 3, 5), (2, 64, 83), (3, 256, 128), (1, 257, 64), (2, 512, 100), (2, 512, 4092 // 31),
    (1, 1024, 40), (1, 1030, 72), (1, 2050, 33), (2, 100, 65), (1, 600, 67), (2, 16, 6, 7), (2, 64, 28, 28), (1, 32, 1, 8),
]


def ln_inputs(shape, dtype, seed, shift):
    g = gen(seed)
    x = randn(g, *shape, dtype=dtype, scale=1.5, shift=shift)
    w = randn(g, shape[1], dtype=dtype, scale=0.3, shift=1.0)
    b = randn(g, shape[1], dtype=dtype, scale=0.3)
    go = randn(g, *shape, dtype=dtype)
    return x, w, b, go


def ln_bound(x, mean, rstd):
    # x - mean: the mean's rounding (16 u of the largest |x|), times rstd; rstd
    # and the products: 16 u relative
    top = x.double().abs().amax(1, keepdim=True)
    m, r = mean.unsqueeze(1), rstd.unsqueeze(1)
    return 16 * U32 * (top * r + ((x.double() - m) * r).abs())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", LN_SHAPES)
def test_layer_norm(shape, dtype):
    print("layer norm", shape, dtype, flush=True)
    x, w, b, go = ln_inputs(shape, dtype, 1, 0.5)
    side = (1, -1) + (1,) * (len(shape) - 2)
    for weight, bias in ((w, b), (None, None), (w, None), (None, b)):
        y, mean, rstd = sequence.layer_norm(x, weight, bias, with_stats=True)
        wy, wm, wr = ref.layer_norm(x, weight, bias)
        e = ln_bound(x, wm, wr)
        top = x.double().abs().amax(1)
        # a variance of nothing (C = 1, or equal values) leaves the rounding of x - mean under eps
        within(mean, wm, 16 * U32 * top, "mean")
        within(rstd, wr, wr * (16 * U32 * (1 + top * wr) ** 2), "rstd")
        bound = e if weight is None else e * weight.double().abs().view(side)
        if bias is not None:
            bound = bound + 4 * U32 * bias.double().abs().view(side)
        bound = bound + (ref.unit(dtype) if dtype == BF16 else 4 * U32) * wy.abs() * 1.01
        within(y, wy, bound, "y")
        assert torch.equal(y, sequence.layer_norm(x, weight, bias))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", LN_SHAPES)
def test_layer_norm_backward(shape, dtype):
    print("layer norm backward", shape, dtype, flush=True)
    x, w, b, go = ln_inputs(shape, dtype, 2, -0.25)
    side = (1, -1) + (1,) * (len(shape) - 2)
    for weight in (w, None):
        _, mean, rstd = sequence.layer_norm(x, weight, None, with_stats=True)
        got = sequence.layer_norm_backward(x, go, mean, rstd, weight)
        want = ref.layer_norm_backward(x, go, weight)
        _, wm, wr = ref.layer_norm(x)
        r = wr.unsqueeze(1)
        xh = (x.double() - wm.unsqueeze(1)) * r
        u = go.double() if weight is None else go.double() * weight.double().view(side)
        # relative errors of xh and rstd: those of the forward
        e = 16 * U32 * (1 + (x.double().abs().amax(1, keepdim=True) * r)) ** 2
        ub = u.abs().mean(1, keepdim=True)
        ux = (u * xh).abs().mean(1, keepdim=True)
        bound = 4 * e * r * (u.abs() + ub + (xh.abs() + 1) * (ux + ub))
        own = ref.unit(dtype) * 1.01
        within(got["x"], want["x"], bound + own * want["x"].abs(), "grad_x")
        rest = [0] + list(range(2, x.dim()))
        n = x.numel() // shape[1]
        # n terms added in runs: at most n u relative to the absolute sum, sqrt(n) of it is far more than is seen
        s = (64 + math.sqrt(n)) * U32
        within(got["weight"], want["weight"], ((e * (xh.abs() + 1) + s * xh.abs()) * go.double().abs()).sum(rest) +
               own * want["weight"].abs(), "grad_weight")
        within(got["bias"], want["bias"], s * go.double().abs().sum(rest) + own * want["bias"].abs(), "grad_bias")
        for need in (("x",), ("weight",), ("bias",), ("weight", "bias"), ()):
            some = sequence.layer_norm_backward(x, go, mean, rstd, weight, need=need)
            assert set(some) == set(need)
            for key in need:
                assert torch.equal(some[key], got[key]), key


def test_layer_norm_large_mean_keeps_digits():
    x = randn(gen(3), 4, 1024, shift=1000.0)
    y, mean, rstd = sequence.layer_norm(x, with_stats=True)
    wy, wm, wr = ref.layer_norm(x)
    within(y, wy, ln_bound(x, wm, wr) + 4 * U32 * wy.abs(), "y")


def test_layer_norm_in_place_and_unaligned():
    for dtype in (F32, BF16):
        for shape in ((6, 512), (2, 64, 96)):
            n = math.prod(shape)
            store = randn(gen(4), n + 1, dtype=dtype)
            x = store[1:].view(shape)  # rows off every alignment
            want = sequence.layer_norm(x.clone())
            within(sequence.layer_norm(x), want.double(), (2 * ref.unit(dtype) + 32 * U32) * (1 + want.double().abs()), "unaligned")
            y = x.clone()
            assert sequence.layer_norm(y, out=y) is y
            assert torch.equal(y, want)


ODD_SHAPES = [
    (9, 1), (6, 5), (5, 9), (7, 15), (3, 65), (6, 513), (5, 1022), (3, 2047), (3, 4099), (2, 8191), (2, 12345), (2, 16383), (2, 16391),
    (3, 6, 2), (2, 9, 7), (2, 1030, 3), (2, 5, 9), (2, 64, 97), (1, 256, 131), (2, 300, 65), (1, 700, 71), (2, 1025, 19), (1, 2051, 37),
    (1, 33, 4093), (3, 65, 641), (1, 33), (77, 40), (301, 101), (70, 200), (4099, 37),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", ODD_SHAPES)
def test_layer_norm_odd_sizes_between_neighbours(shape, dtype):
    # inputs and results that start off every alignment, with other values right before and after
    print("layer norm, odd", shape, dtype, flush=True)
    n, C = math.prod(shape), shape[1]
    side = (1, -1) + (1,) * (len(shape) - 2)

    def amid(t):  # the same values one element off, NaN around them
        store = torch.full((t.numel() + 32,), float("nan"), dtype=t.dtype, device=DEV)
        store[17:17 + t.numel()] = t.reshape(-1)
        return store[17:17 + t.numel()].view(t.shape), store

    x, w, b, go = ln_inputs(shape, dtype, 11, 0.5)
    (ox, sx), (ow, _), (ob, _), (og, _) = amid(x), amid(w), amid(b), amid(go)
    wy, wm, wr = ref.layer_norm(x, w, b)
    e = ln_bound(x, wm, wr)
    bound = e * w.double().abs().view(side) + 4 * U32 * b.double().abs().view(side)
    bound = bound + (ref.unit(dtype) if dtype == BF16 else 4 * U32) * wy.abs() * 1.01
    y, mean, rstd = sequence.layer_norm(ox, ow, ob, with_stats=True)
    within(y, wy, bound, "y")
    within(mean, wm, 16 * U32 * x.double().abs().amax(1), "mean")
    got = sequence.layer_norm_backward(ox, og, mean, rstd, ow)
    want = ref.layer_norm_backward(x, go, w)
    r = wr.unsqueeze(1)
    xh = (x.double() - wm.unsqueeze(1)) * r
    u = go.double() * w.double().view(side)
    e = 16 * U32 * (1 + (x.double().abs().amax(1, keepdim=True) * r)) ** 2
    ub, ux = u.abs().mean(1, keepdim=True), (u * xh).abs().mean(1, keepdim=True)
    own = ref.unit(dtype) * 1.01
    within(got["x"], want["x"], 4 * e * r * (u.abs() + ub + (xh.abs() + 1) * (ux + ub)) + own * want["x"].abs(), "grad_x")
    rest = [0] + list(range(2, x.dim()))
    s = (64 + math.sqrt(n // C)) * U32  # as above
    within(got["weight"], want["weight"], (go.double().abs() * (e * (1 + xh.abs()) + s * xh.abs())).sum(rest) + own * want["weight"].abs(), "grad_weight")
    within(got["bias"], want["bias"], s * go.double().abs().sum(rest) + own * want["bias"].abs(), "grad_bias")
    # in place: the same bits, and nothing around them is touched
    assert sequence.layer_norm(ox, ow, ob, out=ox) is ox
    assert torch.equal(ox, y)
    assert torch.isnan(sx[:17]).all() and torch.isnan(sx[17 + n:]).all()


def test_layer_norm_channels_past_32_bit_offsets():
    # 1025 channels, two threads across a row: channel 255 of 2^22 + 8 float32 positions starts past 2^32 bytes
    C, L = 1025, (1 << 22) + 8
    x = torch.empty((1, C, L), device=DEV)
    for c in range(C):  # a channel at a time, so that no index passes 32 bits in what fills it
        x[0, c].normal_(generator=gen(100 + c))
    at = torch.tensor([0, 1, 7, 8, 1000003, L - 9, L - 1], device=DEV)
    some = torch.stack([x[0, c][at] for c in range(C)]).unsqueeze(0)
    y, mean, rstd = sequence.layer_norm(x, with_stats=True)
    wy, wm, wr = ref.layer_norm(some)
    got = torch.stack([y[0, c][at] for c in range(C)]).unsqueeze(0)
    within(got, wy, ln_bound(some, wm, wr) + 4 * U32 * wy.abs(), "y")
    grad = sequence.layer_norm_backward(x, x, mean, rstd, need=("x",))["x"]
    got = torch.stack([grad[0, c][at] for c in range(C)]).unsqueeze(0)
    # against the same positions by themselves, whose gradients are checked above
    _, m, r = sequence.layer_norm(some, with_stats=True)
    want = sequence.layer_norm_backward(some, some, m, r, need=("x",))["x"].double()
    e = 16 * U32 * (1 + some.double().abs().amax(1, keepdim=True) * wr.unsqueeze(1)) ** 2
    within(got, want, 16 * e * (1 + some.double().abs()) * (1 + wr.unsqueeze(1)), "grad_x")


def test_layer_norm_empty():
    for shape in ((0, 8), (0, 8, 4), (2, 8, 0)):
        x = torch.empty(shape, device=DEV)
        y, mean, rstd = sequence.layer_norm(x, with_stats=True)
        assert y.shape == x.shape and mean.numel() == 0
        grads = sequence.layer_norm_backward(x, torch.empty_like(x), mean, rstd)
        assert not grads["weight"].any() and not grads["bias"].any() and grads["x"].shape == x.shape


@pytest.mark.parametrize("shape", [(6, 24), (2, 24, 9)])
def test_layer_norm_gradient_against_differences(shape):
    x, w, b, go = ln_inputs(shape, F32, 5, 0.5)
    _, mean, rstd = sequence.layer_norm(x, w, b, with_stats=True)
    got = sequence.layer_norm_backward(x, go, mean, rstd, w)
    f = lambda x, w, b: (ref.layer_norm(x, w, b)[0] * go.double()).sum()  # noqa: E731
    at, h = [x.double(), w.double(), b.double()], 1e-4
    for i, key in enumerate(("x", "weight", "bias")):
        d = randn(gen(6 + i), *at[i].shape).double()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * d, at[i] - h * d
        slope = (f(*up) - f(*down)) / (2 * h)
        # differences: h^2 of the third derivative; gradient: 1e-5 of the absolute sum
        size = (got[key].double() * d).abs().sum()
        assert abs(float((got[key].double() * d).sum() - slope)) <= 1e-5 * float(size), key


# ---- rotary -----------------------------------------------------------------------

def rotary_case(seed, B, L, Hq, Hkv, D, sections, dtype, shared=False, P=77):
    g = gen(seed)
    R = sum(sections)
    angle = torch.rand((P, R), generator=g, device=DEV, dtype=torch.float64) * 40 - 20
    cos, sin = angle.cos().float(), angle.sin().float()
    pos = torch.randint(0, P, (1 if shared else B, L, len(sections)), generator=g, device=DEV).int()
    return randn(g, B, L, Hq, D, dtype=dtype), randn(g, B, L, Hkv, D, dtype=dtype), cos, sin, pos


def rotary_bound(x, dtype):
    # two products and their sum: 4 u of |a| + |b| <= 2 max
    return 8 * U32 * x.double().abs().amax(-1, keepdim=True) + (1.01 * 2.0 ** -8 if dtype == BF16 else 0.0) * 2 * x.double().abs().amax(-1, keepdim=True)


ROTARY = [
    (1, 1, 1, 1, 2, (1,)), (2, 3, 2, 1, 64, (32,)), (1, 5, 8, 2, 128, (16, 24, 24)), (2, 33, 3, 3, 80, (13, 27)),
    (3, 7, 5, 1, 64, (8, 8)), (2, 9, 4, 4, 66, (32,)), (1, 4, 2, 2, 31, (5, 0, 4, 6)), (2, 64, 4, 2, 96, (10, 10, 12, 16)),
    (1, 700, 6, 2, 64, (32,)), (2, 17, 9, 1, 100, (33,)),
]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", ROTARY)
def test_rotary(case, interleaved, dtype):
    print("rotary", case, interleaved, dtype, flush=True)
    B, L, Hq, Hkv, D, sections = case
    for shared in (False, True):
        q, k, cos, sin, pos = rotary_case(11, *case, dtype, shared)
        for inverse in (False, True):
            kw = dict(interleaved=interleaved, inverse=inverse)
            a, b = sequence.rotary(q, k, cos, sin, pos, sections, **kw)
            for got, x in ((a, q), (b, k)):
                want = ref.rotary(x, cos, sin, pos, sections, **kw)
                within(got, want, rotary_bound(x, dtype), "rotary")
                assert torch.equal(got[..., 2 * sum(sections):], x[..., 2 * sum(sections):])
            only, none = sequence.rotary(q, None, cos, sin, pos, sections, **kw)
            assert none is None and torch.equal(only, a)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rotary_layouts(dtype):
    B, L, Hq, Hkv, D, sections = 2, 19, 4, 2, 64, (12, 20)
    q, k, cos, sin, pos = rotary_case(12, B, L, Hq, Hkv, D, sections, dtype)
    want = sequence.rotary(q, k, cos, sin, pos, sections)
    # head slices of one buffer, turned in place
    both = torch.cat([q, k, k], 2)
    rest = both[:, :, Hq + Hkv:].clone()
    a, b = both[:, :, :Hq], both[:, :, Hq:Hq + Hkv]
    sequence.rotary(a, b, cos, sin, pos, sections, out=(a, b))
    assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(both[:, :, Hq + Hkv:], rest)
    # heads ahead of positions; rows off every alignment
    qt, kt = q.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(1, 2).contiguous().transpose(1, 2)
    got = sequence.rotary(qt, kt, cos, sin, pos, sections)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    wide = torch.zeros((B, L, Hq, D + 3), dtype=dtype, device=DEV)
    wide[..., 1:D + 1] = q
    got, _ = sequence.rotary(wide[..., 1:D + 1], None, cos, sin, pos, sections)
    within(got, want[0].double(), 2 * rotary_bound(q, dtype), "unaligned")


def test_rotary_positions_outside_the_tables_are_clamped():
    q, k, cos, sin, pos = rotary_case(13, 2, 6, 2, 1, 32, (16,), F32)
    wild = pos.clone()
    wild[0, 0], wild[0, 1], wild[1, 2], wild[1, 3] = -1, cos.shape[0], -2 ** 31, 2 ** 31 - 1
    got, _ = sequence.rotary(q, None, cos, sin, wild, (16,))
    within(got, ref.rotary(q, cos, sin, wild, (16,)), rotary_bound(q, F32), "clamped")


def test_rotary_inverse_is_the_gradient():
    q, k, cos, sin, pos = rotary_case(14, 2, 5, 2, 1, 40, (7, 9), F32)
    g = randn(gen(15), *q.shape)
    for interleaved in (False, True):
        back, _ = sequence.rotary(g, None, cos, sin, pos, (7, 9), interleaved=interleaved, inverse=True)
        d = randn(gen(16), *q.shape).double()
        f = lambda x: (ref.rotary(x, cos, sin, pos, (7, 9), interleaved) * g.double()).sum()  # noqa: E731
        slope = (f(q.double() + d) - f(q.double() - d)) / 2  # linear
        assert abs(float((back.double() * d).sum() - slope)) <= 1e-6 * float((back.double() * d).abs().sum())


def test_rotary_empty():
    q, k, cos, sin, pos = rotary_case(17, 2, 3, 2, 1, 32, (16,), F32)
    a, b = sequence.rotary(q[:, :0], k[:, :0], cos, sin, pos[:, :0].contiguous(), (16,))
    assert a.shape == (2, 0, 2, 32) and b.shape == (2, 0, 1, 32)


# ---- attention ----------------------------------------------------------------------

def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# B, Lq, Lk, Hq, Hkv, D, mask
ATT = [
    (1, 1, 1, 1, 1, 1, {}),
    (1, 1, 1, 1, 1, 64, dict(causal=True)),
    (2, 3, 5, 2, 1, 7, {}),
    (1, 31, 33, 2, 2, 32, dict(causal=True)),
    (2, 64, 64, 4, 2, 64, dict(causal=True)),
    (1, 65, 63, 3, 1, 64, dict(causal=True)),           # the first queries see nothing
    (2, 83, 83, 8, 8, 64, {}),
    (1, 127, 129, 2, 1, 128, dict(causal=True)),
    (1, 128, 128, 1, 1, 128, {}),
    (2, 129, 257, 4, 4, 80, dict(causal=True)),
    (1, 200, 190, 2, 1, 100, dict(window=17)),
    (1, 300, 300, 2, 2, 64, dict(causal=True, window=33)),
    (1, 40, 40, 4, 1, 33, dict(window=1)),
    (3, 50, 70, 2, 1, 64, dict(kv_lens=(70, 0, 13))),   # a batch without keys
    (3, 50, 70, 2, 1, 128, dict(kv_lens=(64, 1, 65), causal=True)),
    (3, 9, 300, 4, 1, 64, dict(kv_lens=(300, 9, 4), causal=True, q_start=(291, 0, -5))),
    (4, 1, 513, 8, 2, 128, dict(kv_lens=(513, 1, 0, 256), causal=True, q_start=(512, 0, -1, 255))),
    (2, 1, 2000, 4, 4, 64, {}),
    (1, 1, 4100, 16, 1, 128, dict(window=1000, causal=True)),
    (2, 2, 1100, 16, 1, 96, dict(causal=True)),
    (2, 5, 700, 6, 2, 64, dict(causal=True, window=100)),
    (1, 33, 5000, 1, 1, 64, dict(causal=True)),
    (1, 100, 30, 2, 1, 64, dict(q_start=(1000,), causal=True)),
    (1, 20, 90, 2, 1, 64, dict(q_start=(-40,), window=30)),
    (1, 20, 90, 2, 1, 64, dict(q_start=(2 ** 31 - 1,), window=30)),  # past every key
    (1, 10, 40, 2, 1, 32, dict(kv_lens=(99,))),          # lengths past the tensor are clamped
    (1, 10, 40, 2, 1, 32, dict(kv_lens=(-3,))),
    (2, 17, 0, 2, 1, 64, {}),                            # no keys at all
]


def mask_of(spec):
    return {k: i32(*v) if isinstance(v, tuple) else v for k, v in spec.items()}


def ref_mask(mask, Lk):
    m = dict(mask)
    if m.get("kv_lens") is not None:
        m["kv_lens"] = m["kv_lens"].clamp(0, Lk)
    return m


def att_inputs(seed, B, Lq, Lk, Hq, Hkv, D, dtype):
    g = gen(seed)
    return (randn(g, B, Lq, Hq, D, dtype=dtype), randn(g, B, Lk, Hkv, D, dtype=dtype), randn(g, B, Lk, Hkv, D, dtype=dtype),
            randn(g, B, Lq, Hq, D, dtype=dtype))


def att_bound(out, spread, dtype):
    # P: 64 u32 (score and exponential) and, in bf16, one rounding; sums: 64 u32;
    # out: one rounding
    up = 64 * U32 + (2.0 ** -8 if dtype == BF16 else 0.0)
    return (up + 64 * U32) * 1.01 * spread + ref.unit(dtype) * 1.01 * out.abs()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", ATT, ids=lambda c: "-".join(str(v) for v in c[:6]) + "-" + "-".join(c[6]))
def test_attention(case, dtype):
    print("attention", case, dtype, flush=True)
    shape, mask = case[:6], mask_of(case[6])
    q, k, v, _ = att_inputs(21, *shape, dtype)
    out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
    wo, wl, spread = ref.attention(q, k, v, **ref_mask(mask, shape[2]))
    within(lse, wl, 64 * U32 * (4 + wl.abs().nan_to_num(0, 0, 0)), "lse")
    within(out, wo, att_bound(wo, spread, dtype), "out")
    assert torch.equal(out, sequence.attention(q, k, v, **mask))
    assert not out[(wl == -math.inf).transpose(1, 2)].any()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("case", ATT, ids=lambda c: "-".join(str(v) for v in c[:6]) + "-" + "-".join(c[6]))
def test_attention_backward(case, dtype):
    print("attention backward", case, dtype, flush=True)
    shape, mask = case[:6], mask_of(case[6])
    q, k, v, g = att_inputs(22, *shape, dtype)
    out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
    got = sequence.attention_backward(q, k, v, out, lse, g, **mask)
    want, bound = ref.attention_backward(q, k, v, g, storage=dtype, **ref_mask(mask, shape[2]))
    for key in "qkv":
        within(got[key], want[key], bound[key] * 1.01 + 1e-30, "grad_" + key)
    for need in (("q",), ("k",), ("v",), ("k", "v")):
        some = sequence.attention_backward(q, k, v, out, lse, g, need=need, **mask)
        assert set(some) == set(need) and all(torch.equal(some[n], got[n]) for n in need)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,mask", [
    ((3, 136, 136, 4, 1, 128), dict(causal=True, kv_lens=(34, 0, 136))),
    ((2, 300, 90, 4, 1, 64), dict(window=70, kv_lens=(90, 17))),
    ((1, 129, 200, 2, 1, 32), dict(causal=True)),
    ((2, 513, 33, 1, 1, 80), dict()),
    ((1, 97, 260, 8, 2, 64), dict(causal=True, window=40)),
])
def test_attention_gradients_in_short_parts(shape, mask, dtype):
    """Few workgroups: the rows of a key tile in parts of 128 or 256, some of them with nothing to do."""
    print("attention gradients in parts", shape, mask, dtype, flush=True)
    mask = dict(mask)
    if "kv_lens" in mask:
        mask["kv_lens"] = torch.tensor(mask["kv_lens"], dtype=torch.int32, device=DEV)
    q, k, v, g = att_inputs(29, *shape, dtype)
    out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
    got = sequence.attention_backward(q, k, v, out, lse, g, **mask)
    want, bound = ref.attention_backward(q, k, v, g, storage=dtype, **ref_mask(mask, shape[2]))
    for key in "qkv":
        within(got[key], want[key], bound[key] * 1.01 + 1e-30, "grad_" + key)
    again = sequence.attention_backward(q, k, v, out, lse, g, **mask)
    assert all(torch.equal(again[key], got[key]) for key in "qkv")


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_attention_larger(dtype):
    """Several tiles of keys and rows per workgroup, and split gradients."""
    for shape, mask in (((2, 700, 1500, 4, 1, 128), dict(causal=True)), ((1, 1024, 1024, 8, 2, 64), dict(causal=True, window=300))):
        print("attention larger", shape, mask, dtype, flush=True)
        q, k, v, g = att_inputs(23, *shape, dtype)
        out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
        wo, wl, spread = ref.attention(q, k, v, **mask)
        within(out, wo, att_bound(wo, spread, dtype), "out")
        got = sequence.attention_backward(q, k, v, out, lse, g, **mask)
        want, bound = ref.attention_backward(q, k, v, g, storage=dtype, **mask)
        for key in "qkv":
            within(got[key], want[key], bound[key] * 1.01, "grad_" + key)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(2, 70, 90, 4, 2, 64), (2, 1, 600, 4, 2, 64), (1, 40, 40, 2, 1, 20)])
def test_attention_layouts(shape, dtype):
    """Slices of one projection's output, heads ahead of positions, storage off
    every alignment, and a key head repeated by a stride of 0: the same bits
    as contiguous inputs, in and out."""
    B, Lq, Lk, Hq, Hkv, D = shape
    q, k, v, g = att_inputs(24, *shape, dtype)
    out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
    grads = sequence.attention_backward(q, k, v, out, lse, g, causal=True)

    def check(q, k, v, g, o, gq, gk, gv, exact):
        same = torch.equal if exact else lambda a, b: torch.allclose(a.float(), b.float(), rtol=2 * ref.unit(dtype), atol=1e-5)
        assert same(sequence.attention(q, k, v, causal=True, out=o), out)
        some = sequence.attention_backward(q, k, v, o, lse, g, causal=True, grads={"q": gq, "k": gk, "v": gv})
        assert some["q"] is gq and same(gq, grads["q"]) and same(gk, grads["k"]) and same(gv, grads["v"])

    kv = torch.zeros((B, Lk, 2 * Hkv + 1, D), dtype=dtype, device=DEV)
    kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv] = k, v
    gkv = torch.full_like(kv, 3.0)
    check(q, kv[:, :, :Hkv], kv[:, :, Hkv:2 * Hkv], g, torch.empty_like(q), torch.empty_like(q), gkv[:, :, :Hkv],
          gkv[:, :, Hkv:2 * Hkv], True)
    assert (gkv[:, :, 2 * Hkv:] == 3.0).all()
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    check(t(q), t(k), t(v), t(g), t(torch.empty_like(q)), t(torch.empty_like(q)), t(torch.empty_like(k)), t(torch.empty_like(k)), True)

    def off(x):
        wide = torch.zeros(x.shape[:3] + (D + 3,), dtype=dtype, device=DEV)
        wide[..., 1:D + 1] = x
        return wide[..., 1:D + 1]

    check(off(q), off(k), off(v), off(g), off(q), off(q), off(k), off(v), False)
    one = sequence.attention(q, k[:, :, :1].expand_as(k), v[:, :, :1].expand_as(v), causal=True)
    assert torch.equal(one, sequence.attention(q, k[:, :, :1].repeat(1, 1, Hkv, 1), v[:, :, :1].repeat(1, 1, Hkv, 1), causal=True))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Lq", [1, 40])
def test_attention_ignores_what_lies_past_the_lengths(Lq, dtype):
    B, Lk, Hq, Hkv, D = 3, 300, 4, 2, 64
    q, k, v, g = att_inputs(25, B, Lq, Lk, Hq, Hkv, D, dtype)
    lens = i32(300, 133, 0)
    kw = dict(kv_lens=lens, q_start=lens - Lq, causal=True)
    out, lse = sequence.attention(q, k, v, with_lse=True, **kw)
    grads = sequence.attention_backward(q, k, v, out, lse, g, **kw)
    past = (torch.arange(Lk, device=DEV).view(1, Lk) >= lens.view(B, 1))
    for junk in (float("nan"), float("inf"), -float("inf"), torch.finfo(dtype).min):
        kj, vj = k.clone(), v.clone()
        kj[past], vj[past] = junk, junk
        o2, l2 = sequence.attention(q, kj, vj, with_lse=True, **kw)
        assert torch.equal(o2, out) and torch.equal(l2, lse)
        g2 = sequence.attention_backward(q, kj, vj, out, lse, g, **kw)
        assert all(torch.equal(g2[n], grads[n]) for n in "qkv")
    assert not grads["k"][past].any() and not grads["v"][past].any()


def test_attention_extreme_scores():
    """Scores far apart (one key takes all), and far below zero (no underflow of the sum)."""
    B, L, H, D = 1, 96, 2, 64
    q, k, v, _ = att_inputs(26, B, L, L, H, H, D, F32)
    for qs, ks in ((q * 30, k * 30), (q.abs() * 10, -k.abs() * 10)):
        out, lse = sequence.attention(qs, ks, v, with_lse=True)
        wo, wl, spread = ref.attention(qs, ks, v)
        # the scores' rounding grows with their terms: 64 u of scale * sum |q k|
        big = float(torch.einsum("blhd,bmhd->bhlm", qs.double().abs(), ks.double().abs()).max()) / math.sqrt(D)
        within(lse, wl, 4 * U32 * big, "lse")
        within(out, wo, 16 * U32 * big * spread + 1e-6, "out")


def test_attention_nan_reaches_its_row_only():
    q, k, v, _ = att_inputs(27, 1, 70, 70, 2, 2, 64, BF16)
    clean = sequence.attention(q, k, v)
    q[0, 33, 1, 5] = float("nan")
    out = sequence.attention(q, k, v)
    assert out[0, 33, 1].isnan().all()
    out[0, 33, 1] = clean[0, 33, 1]
    assert torch.equal(out, clean)


@pytest.mark.parametrize("mask", [{}, dict(causal=True), dict(causal=True, window=9), dict(kv_lens=(31, 0))])
def test_attention_gradient_against_differences(mask):
    B, Lq, Lk, Hq, Hkv, D = 2, 19, 37, 4, 2, 24
    mask = mask_of(mask)
    q, k, v, g = att_inputs(28, B, Lq, Lk, Hq, Hkv, D, F32)
    out, lse = sequence.attention(q, k, v, with_lse=True, **mask)
    got = sequence.attention_backward(q, k, v, out, lse, g, **mask)
    at, h = [q.double(), k.double(), v.double()], 1e-4
    f = lambda *a: (ref.attention(*a, **mask)[0] * g.double()).sum()  # noqa: E731
    for i, key in enumerate("qkv"):
        d = randn(gen(29 + i), *at[i].shape).double()
        up, down = list(at), list(at)
        up[i], down[i] = at[i] + h * d, at[i] - h * d
        slope = (f(*up) - f(*down)) / (2 * h)
        assert abs(float((got[key].double() * d).sum() - slope)) <= 1e-5 * float((got[key].double() * d).abs().sum()), key


def test_attention_scale():
    q, k, v, _ = att_inputs(31, 1, 20, 30, 2, 1, 64, F32)
    out = sequence.attention(q, k, v, scale=0.3)
    wo, _, spread = ref.attention(q, k, v, scale=0.3)
    within(out, wo, 3 * att_bound(wo, spread, F32), "out")  # scores 2.4 times the usual


@pytest.mark.parametrize("Lq", [1, 130])
def test_attention_offsets_past_32_bits(Lq):
    """A cache whose second sequence and last positions lie past 2^31 elements."""
    Lk, D = 200, 64
    row = (1 << 31) // 150 // 8 * 8  # position 151 starts past 2^31
    store = torch.zeros(row * Lk + D, dtype=BF16, device=DEV)
    q, k, v, g = att_inputs(32, 1, Lq, Lk, 1, 1, D, BF16)
    far = store.as_strided((1, Lk, 1, D), (0, row, 0, 1))
    far.copy_(k)
    out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
    assert torch.equal(sequence.attention(q, far, v, causal=True), out)
    assert torch.equal(sequence.attention(q, k, far, causal=True), sequence.attention(q, k, k, causal=True))
    want = sequence.attention_backward(q, k, v, out, lse, g, causal=True)
    got = sequence.attention_backward(q, far, v, out, lse, g, causal=True)
    assert all(torch.equal(got[n], want[n]) for n in "qkv")
    sequence.attention_backward(q, k, v, out, lse, g, causal=True, need=("k",), grads={"k": far})
    assert torch.equal(far, want["k"])


def test_attention_empty():
    for B, Lq, Lk in ((0, 4, 4), (2, 0, 5)):
        q, k, v, g = att_inputs(33, B, Lq, Lk, 2, 1, 64, BF16)
        out, lse = sequence.attention(q, k, v, with_lse=True)
        assert out.shape == q.shape and lse.shape == (B, 2, Lq)
        grads = sequence.attention_backward(q, k, v, out, lse, g)
        assert not grads["k"].any() and not grads["v"].any() and grads["q"].shape == q.shape


# ---- all of them ------------------------------------------------------------------------

def every_operator(seed, dtype, Lq=150):
    x, w, b, go = ln_inputs((4, 256, 72), dtype, seed, 0.5)
    rows = ln_inputs((50, 1024), dtype, seed, 0.5)
    rq, rk, cos, sin, pos = rotary_case(seed, 2, 40, 4, 2, 64, (12, 20), dtype)
    q, k, v, g = att_inputs(seed, 2, Lq, 900, 4, 2, 64, dtype)

    def call():
        y, mean, rstd = sequence.layer_norm(x, w, b, with_stats=True)
        out, lse = sequence.attention(q, k, v, causal=True, with_lse=True)
        step, _ = sequence.attention(q[:, :1].contiguous(), k, v, with_lse=True)
        y2, m2, r2 = sequence.layer_norm(rows[0], rows[1], rows[2], with_stats=True)
        return [y, mean, rstd, *sequence.layer_norm_backward(x, go, mean, rstd, w).values(), y2,
                *sequence.layer_norm_backward(rows[0], rows[3], m2, r2, rows[1]).values(),
                *sequence.rotary(rq, rk, cos, sin, pos, (12, 20)), out, lse, step,
                *sequence.attention_backward(q, k, v, out, lse, g, causal=True).values()]

    return call


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_repeats_bit_for_bit(dtype):
    call = every_operator(41, dtype)
    first = [t.clone() for t in call()]
    for _ in range(4):
        for a, b in zip(first, call()):
            assert torch.equal(a, b)


def test_another_stream():
    """Work follows torch's current stream, with a workspace of that stream's own."""
    call = every_operator(42, BF16)
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call()
        done = side.record_event()
    done.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_graph_replays():
    call = every_operator(43, BF16)
    want = [t.clone() for t in call()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()  # sizes the workspace of this stream
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        call()
        torch.cuda.synchronize()


# ---- refusals ---------------------------------------------------------------------------

def test_refusals():
    x = torch.zeros((2, 8, 4), device=DEV)
    bad = dc1d.Dc1dValueError

    def refused(status, fn, *a, **kw):
        with pytest.raises(bad) as e:
            fn(*a, **kw)
        assert e.value.status == status

    refused(dc1d.ERR_BAD_DTYPE, sequence.layer_norm, x.half())
    refused(dc1d.ERR_BAD_DTYPE, sequence.layer_norm, x, torch.ones(8, dtype=BF16, device=DEV))
    refused(dc1d.ERR_BAD_SHAPE, sequence.layer_norm, x, torch.ones(7, device=DEV))
    refused(dc1d.ERR_BAD_SHAPE, sequence.layer_norm, torch.zeros(8, device=DEV))
    refused(dc1d.ERR_BAD_ARG, sequence.layer_norm, x, eps=-1.0)
    refused(dc1d.ERR_BAD_ARG, sequence.layer_norm, x, eps=float("nan"))
    with pytest.raises(ValueError):
        sequence.layer_norm(x.transpose(0, 1))
    with pytest.raises(ValueError):
        sequence.layer_norm(x.cpu())
    with pytest.raises(ValueError):
        sequence.layer_norm(x, torch.ones(8))
    q = torch.zeros((2, 3, 4, 64), device=DEV)
    k = torch.zeros((2, 5, 2, 64), device=DEV)
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention, q, k, k[:, :4])
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention, q[:, :, :3], k, k)
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention, q[..., ::2], k[..., ::2], k[..., ::2])
    big = torch.zeros((1, 1, 1, 129), device=DEV)
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention, big, big, big)
    refused(dc1d.ERR_BAD_DTYPE, sequence.attention, q, k.bfloat16(), k)
    refused(dc1d.ERR_BAD_DTYPE, sequence.attention, q, k, k, kv_lens=torch.zeros(2, dtype=torch.int64, device=DEV))
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention, q, k, k, kv_lens=i32(1, 2, 3))
    refused(dc1d.ERR_BAD_ARG, sequence.attention, q, k, k, window=-1)
    for scale in (0.0, -1.0, float("nan"), float("inf"), 1e-300):
        refused(dc1d.ERR_BAD_ARG, sequence.attention, q, k, k, scale=scale)
    refused(dc1d.ERR_ALIAS, sequence.attention, q, k, k, out=q)
    refused(dc1d.ERR_ALIAS, sequence.attention, q, k, k, out=q[:1].expand_as(q))
    long = torch.zeros((1, 4096, 2, 64), device=DEV)
    refused(dc1d.ERR_WORKSPACE, sequence.attention, q[:1, :1], long, long, workspace=torch.zeros(64, dtype=torch.uint8, device=DEV))
    out, lse = sequence.attention(q, k, k, with_lse=True)
    refused(dc1d.ERR_ALIAS, sequence.attention_backward, q, k, k, out, lse, q, grads={"k": k})
    refused(dc1d.ERR_BAD_SHAPE, sequence.attention_backward, q, k, k, out, lse[:1].contiguous(), q)
    cos = torch.zeros((9, 32), device=DEV)
    pos = torch.zeros((2, 3, 1), dtype=torch.int32, device=DEV)
    refused(dc1d.ERR_BAD_ARG, sequence.rotary, q, None, cos, cos, pos, ())
    refused(dc1d.ERR_BAD_ARG, sequence.rotary, q, None, cos, cos, pos, (40,))
    refused(dc1d.ERR_BAD_SHAPE, sequence.rotary, q, None, cos, cos, pos, (30,))
    refused(dc1d.ERR_BAD_SHAPE, sequence.rotary, q, None, cos, cos, pos, (16, 16))
    refused(dc1d.ERR_BAD_DTYPE, sequence.rotary, q, None, cos, cos, pos.long(), (32,))
    refused(dc1d.ERR_ALIAS, sequence.rotary, q, None, cos, cos, pos, (32,), out=(q[:1].expand_as(q), None))
