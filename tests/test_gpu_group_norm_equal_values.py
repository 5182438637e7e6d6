"""Group norm's means: those of equal values are the values themselves, whatever
the order of the sums, so that a constant group gives exactly its bias and no
gradient of its weight; and a mean far from 0 is off by its own rounding only.

u = 2^-24.  The first mean m0 of values v is off by up to K = 100 roundings, j
units of v's last place; x - m0 is then exact, and so are sums of n equal ones
below 2^24 of those units (j n here: 100 x 65536 at the most that a workgroup
holds; what is seen is 16 x 65536), and m0 + (v - m0) = v.  The squares about m0
leave a variance of at most K u (K u v)^2 beside eps.
"""
import pytest
import torch

from deformable_convolution_amd import sequence

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U, K, EPS = 2.0 ** -24, 100, 1e-5
VALUES = [0.1, 0.7, 1000.1, -37.3]

# A group's lanes in one wave; several rows of whole pieces (up to 16 a thread); one odd group a slab; several odd groups.
HELD = [((50, 512), 4), ((2, 784, 64), 4), ((4, 4096, 512), 32), ((70, 890), 1), ((3, 4092, 255), 17), ((3, 257, 255), 17), ((2, 100, 510), 34)]

# Samples in parts: their statistics joined by every workgroup or by a kernel, every group in a tile or channels folded into
# groups, one channel a group, parts that one workgroup reads in several batches.
PARTS = [((2, 5000, 64), 1), ((2, 3000, 264), 3), ((3, 1300, 512), 512), ((2, 6000, 96), 96), ((1, 4100, 1030), 2), ((1, 300, 5000), 1),
         ((2, 700, 4104), 54), ((1, 30000, 8), 1), ((520, 601, 36), 1), ((1, 16384, 257), 1)]


def constant(shape, groups, value, dtype):
    """Every group of equal values, each another one."""
    C = shape[-1]
    per = (torch.tensor(value) * (1 + 0.37 * torch.arange(groups))).to(dtype)
    return per.repeat_interleave(C // groups).expand(shape).contiguous().to(DEV), per.float().to(DEV)


def check_equal(shape, groups, dtype):
    g = torch.Generator().manual_seed(1)
    C = shape[-1]
    w, b = ((torch.randn(C, generator=g) * 0.3 + s).to(dtype).to(DEV) for s in (1.0, 0.0))
    go = torch.randn(shape, generator=g).to(dtype).to(DEV)
    lens = torch.full(shape[:1], shape[1] - 1, dtype=torch.int32, device=DEV) if len(shape) == 3 else None
    for value in VALUES:
        x, per = constant(shape, groups, value, dtype)
        y, mean, rstd = sequence.group_norm(x, groups, w, b, eps=EPS, with_stats=True)
        print(shape, groups, dtype, value, "largest y - bias %.3g" % float((y - b).abs().max()), flush=True)
        assert torch.equal(mean, per.expand(shape[0], groups)) and torch.equal(y, b.expand(shape))
        left = K * U * (K * U * per.abs().double()) ** 2 / (2 * EPS)
        assert ((rstd.double() * EPS ** 0.5 - 1).abs() <= left + 4 * U).all()
        got = sequence.group_norm_backward(x, groups, go, mean, rstd, w, b, need=("weight",))
        assert not got["weight"].any()
        if lens is not None:
            y, mean, _ = sequence.group_norm(x, groups, w, b, eps=EPS, lens=lens, with_stats=True)
            assert torch.equal(mean, per.expand(shape[0], groups)) and torch.equal(y[:, :-1], b.expand(shape)[:, :-1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", HELD)
def test_held(shape, groups, dtype):
    check_equal(shape, groups, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", PARTS)
def test_in_parts(shape, groups, dtype):
    """Every mean is one of its terms and the mean of the differences from it, all of them 0."""
    check_equal(shape, groups, dtype)


@pytest.mark.parametrize("shape,groups", HELD)
def test_mean_far_from_zero(shape, groups):
    """Values about 1000.1: off by the mean's own rounding, and by K roundings of the sum of what is left of them."""
    x = (torch.randn(shape, generator=torch.Generator().manual_seed(2)) * 0.1 + 1000.1).to(DEV)
    _, mean, _ = sequence.group_norm(x, groups, with_stats=True)
    v = x.cpu().double().view(shape[0], -1, groups, shape[-1] // groups)
    want = v.mean((1, 3))
    left = (v - want[:, None, :, None]).abs().amax((1, 3)) + K * U * want.abs()
    assert ((mean.cpu().double() - want).abs() <= U * want.abs() + K * U * left).all()


@pytest.mark.parametrize("shape,groups", [((3, 64), 4), ((2, 30, 32), 4), ((2, 30, 30), 6)])
def test_infinite_values_keep_their_mean(shape, groups):
    """The mean of values of which one is infinite is infinite; what it leaves of the others is NaN, in its group only."""
    x = torch.randn(shape, generator=torch.Generator().manual_seed(3)).to(DEV)
    want, means, _ = sequence.group_norm(x, groups, with_stats=True)
    D = shape[-1] // groups
    x.view(shape[0], -1, shape[-1])[1, 0, D] = float("inf")
    y, mean, rstd = sequence.group_norm(x, groups, with_stats=True)
    assert mean[1, 1] == float("inf") and rstd[1, 1].isnan()
    assert y[1].reshape(-1, shape[-1])[:, D:2 * D].isnan().all()
    y[1].view(-1, shape[-1])[:, D:2 * D] = want[1].view(-1, shape[-1])[:, D:2 * D]
    mean[1, 1] = means[1, 1]
    assert torch.equal(y, want) and torch.equal(mean, means)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape,groups", HELD + PARTS)
def test_squares_past_32_bits(shape, groups, dtype):
    """Values of 1e25, whose squares 32 bits do not hold: the variance is infinite, rstd 0 and y the bias, the mean as ever;
    equal ones of 1e30 have their own as mean."""
    g = torch.Generator().manual_seed(4)
    b = torch.randn(shape[-1], generator=g).to(dtype).to(DEV)
    lens = torch.full(shape[:1], shape[1] - 3, dtype=torch.int32, device=DEV) if len(shape) == 3 else None
    n = shape[1] if lens is None else shape[1] - 3
    part = (lambda t: t) if lens is None else (lambda t: t[:, :n])  # noqa: E731
    spread = torch.randn(shape, generator=g)
    for x in (spread * 1e25, (1 + 0.01 * spread) * 1e30):
        x = x.to(dtype).to(DEV)
        y, mean, rstd = sequence.group_norm(x, groups, None, b, lens=lens, with_stats=True)
        v = part(x).double().view(shape[0], -1, groups, shape[-1] // groups)
        assert not rstd.any() and torch.equal(part(y), part(b.expand(shape)))
        top = v.abs().amax((1, 2, 3)).view(-1, 1)
        assert ((mean.double() - v.mean((1, 3))).abs() <= 320 * U * top).all()  # 320: the most roundings of a shape in parts
    x.fill_(1e30)
    y, mean, rstd = sequence.group_norm(x, groups, None, b, lens=lens, with_stats=True)
    assert (mean == x.view(-1)[0].float()).all() and torch.equal(part(y), part(b.expand(shape)))
