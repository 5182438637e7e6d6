"""Which outputs count as overlapping (no GPU needed: host validation, fake
pointers).  Tensors that are slices of one buffer at the same strides are told
apart exactly, against every element's address; whatever shares memory is
refused."""
import ctypes
import itertools
import random

import numpy as np
import pytest
import torch

from deformable_convolution_amd import dc1d
from test_sequence_boundary import BASE, F32, S, attb, lib, ref, rot  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.device_count() > 0, reason="calls that pass would run on fake pointers")

REACHED = dc1d.ERR_DEVICE  # every check passed


def addresses(t):
    at = np.zeros(1, dtype=np.int64)
    for n, s in zip(t.shape, t.stride):
        at = (at[:, None] + np.arange(n) * s).reshape(-1)
    return at * 4 + t.data


def overlap(a, b):
    return np.intersect1d(addresses(a), addresses(b)).size > 0


def part(buffer_shape, index, slot=9):
    """The view buffer[index] of a contiguous buffer, as a descriptor."""
    t = torch.empty(buffer_shape, device="meta")[index]
    return S(list(t.shape), 0, stride=list(t.stride()), addr=BASE + (slot << 26) + 4 * t.storage_offset())


ALL = slice(None)
PACKED = {  # q, k, v of [2, 7, 2, 64] in one buffer
    "after the positions": ((2, 7, 3, 2, 64), lambda i: (ALL, ALL, i)),
    "after the heads": ((2, 7, 2, 3, 64), lambda i: (ALL, ALL, ALL, i)),
    "in the rows": ((2, 7, 2, 3 * 64), lambda i: (ALL, ALL, ALL, slice(64 * i, 64 * i + 64))),
    "after the batches": ((2, 3, 7, 2, 64), lambda i: (ALL, i)),
    "ahead of the batches": ((3, 2, 7, 2, 64), lambda i: (i,)),
    "along the positions": ((2, 21, 2, 64), lambda i: (ALL, slice(7 * i, 7 * i + 7))),
    "every third position": ((2, 21, 2, 64), lambda i: (ALL, slice(i, None, 3))),
}


@pytest.mark.parametrize("how", PACKED)
def test_packed_tensors(lib, how):  # noqa: F811
    shape, index = PACKED[how]
    p = [part(shape, index(i)) for i in range(3)]
    q = S([2, 7, 2, 64], 0)
    o = S([2, 7, 2, 64], 5)
    other = dict(q=q, out=o, g=S([2, 7, 2, 64], 7), lse=dc1d_lse())
    assert attb(lib, gq=p[0], gk=p[1], gv=p[2], **other) == REACHED
    assert attb(lib, gq=p[0], gk=p[1], gv=p[1], **other) == dc1d.ERR_ALIAS
    assert attb(lib, **{**other, "q": p[0]}, gq=p[0], gk=p[1], gv=p[2]) == dc1d.ERR_ALIAS
    # turned in place
    tables = dict(cos=T2(9, 32), sin=T2(9, 32, 3), pos=T3(2, 7, 2))
    assert rot(lib, q=p[0], k=p[1], qo=p[0], ko=p[1], **tables) == REACHED
    assert rot(lib, q=p[0], k=p[1], qo=p[1], ko=p[0], **tables) == dc1d.ERR_ALIAS


def dc1d_lse():
    from test_sequence_boundary import T
    return T([2, 2, 7], 6)


def T2(a, b, slot=2):
    from test_sequence_boundary import T
    return T([a, b], slot)


def T3(a, b, c):
    from test_sequence_boundary import I32, T
    return T([a, b, c], 4, I32)


def test_against_every_address(lib):  # noqa: F811
    rng = random.Random(5)
    counts = {True: 0, False: 0}
    q, k = S([2, 7, 2, 64], 0), S([2, 7, 2, 64], 1)
    for _ in range(4000):
        B, L, H, D = (rng.choice([1, 2, 2, 3]) for _ in range(4))
        # strides of a buffer with room between the dimensions, in any order
        order = rng.sample(range(3), 3)
        stride, at = [0, 0, 0, 1], D + rng.randint(0, 2 * D)
        for i in order:
            stride[i] = at
            at = at * (B, L, H)[i] + rng.choice([0, 0, rng.randint(0, 2 * at)])
        shape, gap = [B, L, H, D], rng.randint(-at, at)
        gk = S(shape, 0, stride=stride, addr=BASE + (9 << 26))
        gv = S(shape, 0, stride=stride, addr=BASE + (9 << 26) + 4 * gap)
        small = [S(shape, i) for i in (0, 1, 2, 5, 7)]
        from test_sequence_boundary import T
        got = attb(lib, q=small[0], k=small[1], v=small[2], out=small[3], g=small[4], lens=None, lse=T([B, H, L], 6), gq=None, gk=gk, gv=gv)
        want = overlap(gk, gv)
        counts[want] += 1
        assert got == (dc1d.ERR_ALIAS if want else REACHED), (shape, stride, gap)
    assert min(counts.values()) > 500, counts


def test_nothing_that_shares_memory_passes(lib):  # noqa: F811
    """Any strides, not only equal ones: refusing is allowed, accepting an overlap is not."""
    from test_sequence_boundary import T
    rng = random.Random(6)
    accepted = 0
    for _ in range(4000):
        B, L, H, D = (rng.choice([1, 2, 3]) for _ in range(4))
        Hk = rng.choice([h for h in (1, 2, 3) if H % h == 0])

        def some(shape):
            n = [rng.randint(0, 40) for _ in range(3)] + [1]
            return S(shape, 0, stride=n, addr=BASE + (9 << 26) + 4 * rng.randint(0, 60))

        gq, gk = some([B, L, H, D]), some([B, L, Hk, D])
        t = dict(q=S([B, L, H, D], 0), k=S([B, L, Hk, D], 1), v=S([B, L, Hk, D], 2), out=S([B, L, H, D], 5), g=S([B, L, H, D], 7))
        got = attb(lib, lens=None, lse=T([B, H, L], 6), gq=gq, gk=gk, gv=None, **t)
        if got == REACHED:
            accepted += 1
            assert not overlap(gq, gk), (list(gq.shape), list(gq.stride), list(gk.shape), list(gk.stride))
            for g in (gq, gk):
                assert np.unique(addresses(g)).size == addresses(g).size
        else:
            assert got == dc1d.ERR_ALIAS
    assert accepted > 50, accepted
