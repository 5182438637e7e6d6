"""Host-side checks of group norm's and the gated recurrence's C ABI (no GPU
needed): every malformed call is rejected with the documented status before
any device work.  Data pointers are fake: host validation never dereferences
them, and calls that pass every check are made only where no device is
visible."""
import ctypes

import pytest
import torch

from deformable_convolution_amd import dc1d, sequence

BASE, STEP = 0x10000000, 1 << 26
F32, BF16, I32 = 0, 1, 2
BIG = 1 << 62


class Strided(ctypes.Structure):  # dc1d_strided
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


@pytest.fixture(scope="module")
def lib():
    lib = dc1d.load_library()
    p, n, i32, i64, f64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_double
    for name, args in {
            "dc1d_group_norm_workspace_bytes": [p, i64, p],
            "dc1d_group_norm": [p] * 7 + [i64, f64, i32, p, n, p],
            "dc1d_group_norm_backward_workspace_bytes": [p, i64, i32, p],
            "dc1d_group_norm_backward": [p] * 10 + [i64, i32, p, n, p],
            "dc1d_gated_recurrence_workspace_bytes": [p, p],
            "dc1d_gated_recurrence": [p] * 7 + [i32, i32, p, n, p],
            "dc1d_gated_recurrence_backward_workspace_bytes": [p, p],
            "dc1d_gated_recurrence_backward": [p] * 9 + [i32, i32, p, n, p]}.items():
        getattr(lib, name).argtypes = args
    return lib


def T(shape, slot, dtype=F32, addr=None):
    d = dc1d._Tensor()
    d.data = BASE + slot * STEP if addr is None else (addr or None)
    d.dtype, d.ndim = dtype, len(shape)
    d.shape[:min(len(shape), 4)] = shape[:4]
    return d


def S(shape, slot, dtype=F32, stride=None, addr=None, ndim=3):
    d = Strided()
    d.data = BASE + slot * STEP if addr is None else (addr or None)
    d.dtype, d.ndim = dtype, ndim
    d.shape[:] = (list(shape) + [0])[:4]
    d.stride[:] = (list(stride or (max(shape[1], 1) * max(shape[2], 1) if max(shape) < BIG else 1, max(shape[2], 1), 1)) + [0])[:4]
    return d


def ref(t):
    return None if t is None else ctypes.byref(t)


def no_device():
    return torch.cuda.device_count() == 0


X = [3, 10, 12]


def gn(lib, groups=4, eps=1e-5, act=0, ws=(None, 0), **over):
    t = dict(x=T(X, 0), w=T([12], 1), b=T([12], 2), lens=T([3], 3, I32), y=T(X, 4), mean=T([3, 4], 5), rstd=T([3, 4], 6))
    t.update(over)
    return lib.dc1d_group_norm(*[ref(t[k]) for k in ("x", "w", "b", "lens", "y", "mean", "rstd")], groups, eps, act, *ws, None)


def test_group_norm(lib):
    if no_device():
        for over in ({}, dict(w=None, b=None, lens=None, mean=None, rstd=None), dict(y=T(X, 0))):
            assert gn(lib, **over) == dc1d.ERR_DEVICE
        for shape in ([3, 12], [3, 2, 5, 12], [3, 0, 12]):
            assert gn(lib, x=T(shape, 0), y=T(shape, 4), lens=None, act=2) == dc1d.ERR_DEVICE
    for k in ("x", "y"):
        assert gn(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    for k, shape, dt in (("w", [12], F32), ("x", X, F32), ("y", X, F32), ("lens", [3], I32), ("mean", [3, 4], F32)):
        assert gn(lib, **{k: T(shape, 1, dt, addr=0)}) == dc1d.ERR_NULL_PTR
    for over in (dict(x=T(X, 0, 7)), dict(x=T(X, 0, I32)), dict(w=T([12], 1, BF16)), dict(y=T(X, 4, BF16)), dict(mean=T([3, 4], 5, BF16)),
                 dict(lens=T([3], 3, F32))):
        assert gn(lib, **over) == dc1d.ERR_BAD_DTYPE
    for shape in ([12], [3, 10, 0], [3, 10, (1 << 24) + 4], [BIG, 10, 12], [3, BIG, 12], [-1, 10, 12], [3, -1, 12], [1 << 31, 1, 12],
                  [1 << 16, 1 << 15, 12], [BIG, BIG, BIG, 12], [2, 2, 2, 2, 12], [1 << 30, 1, 4]):
        assert gn(lib, x=T(shape, 0)) == dc1d.ERR_BAD_SHAPE, shape
    for over in (dict(y=T([3, 10, 13], 4)), dict(y=T([30, 12], 4)), dict(w=T([4], 1)), dict(b=T([1, 12], 2)), dict(lens=T([4], 3, I32)),
                 dict(lens=T([3, 1], 3, I32)), dict(mean=T([3, 12], 5)), dict(rstd=T([3], 6)),
                 dict(x=T([3, 12], 0), y=T([3, 12], 4)), dict(x=T([3, 2, 5, 12], 0), y=T([3, 2, 5, 12], 4))):  # lens with [B, L, C] only
        assert gn(lib, **over) == dc1d.ERR_BAD_SHAPE, over
    for groups in (0, -1, 5, 13, 24, BIG):
        assert gn(lib, groups) == dc1d.ERR_BAD_ARG
    for eps in (-1e-9, float("nan"), float("inf")):
        assert gn(lib, eps=eps) == dc1d.ERR_BAD_ARG
    for act in (-1, 3, 1 << 30):
        assert gn(lib, act=act) == dc1d.ERR_BAD_ARG
    for over in (dict(y=T(X, 0, addr=BASE + 4)), dict(y=T(X, 1)), dict(y=T(X, 3)), dict(mean=T([3, 4], 6)), dict(rstd=T([3, 4], 0)),
                 dict(mean=T([3, 4], 4)), dict(mean=T([3, 4], 3))):
        assert gn(lib, **over) == dc1d.ERR_ALIAS, over
    n = ctypes.c_size_t()
    assert lib.dc1d_group_norm_workspace_bytes(ref(T(X, 0)), 4, None) == dc1d.ERR_NULL_PTR
    assert lib.dc1d_group_norm_workspace_bytes(None, 4, ctypes.byref(n)) == dc1d.ERR_NULL_PTR
    assert lib.dc1d_group_norm_workspace_bytes(ref(T(X, 0)), 5, ctypes.byref(n)) == dc1d.ERR_BAD_ARG


def gnb(lib, groups=4, act=1, ws=(None, 0), **over):
    t = dict(x=T(X, 0), w=T([12], 1), b=T([12], 2), lens=T([3], 3, I32), g=T(X, 4), mean=T([3, 4], 5), rstd=T([3, 4], 6), gx=T(X, 7),
             gw=T([12], 8), gb=T([12], 9))
    t.update(over)
    return lib.dc1d_group_norm_backward(*[ref(t[k]) for k in ("x", "w", "b", "lens", "g", "mean", "rstd", "gx", "gw", "gb")], groups, act,
                                        *ws, None)


def test_group_norm_backward(lib):
    if no_device():
        for over in ({}, dict(w=None, b=None, lens=None, gw=None, gb=None), dict(gx=T(X, 4)), dict(gx=None)):
            assert gnb(lib, **over) == dc1d.ERR_DEVICE
    for k in ("x", "g", "mean", "rstd"):
        assert gnb(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    assert gnb(lib, gx=T(X, 7, addr=0)) == dc1d.ERR_NULL_PTR
    for over in (dict(g=T(X, 4, BF16)), dict(gw=T([12], 8, BF16)), dict(mean=T([3, 4], 5, I32)), dict(lens=T([3], 3, BF16))):
        assert gnb(lib, **over) == dc1d.ERR_BAD_DTYPE
    for over in (dict(g=T([3, 10, 11], 4)), dict(gx=T([3, 12], 7)), dict(gb=T([13], 9)), dict(rstd=T([4, 3], 6)), dict(lens=T([2], 3, I32))):
        assert gnb(lib, **over) == dc1d.ERR_BAD_SHAPE
    assert gnb(lib, 7) == dc1d.ERR_BAD_ARG and gnb(lib, act=3) == dc1d.ERR_BAD_ARG
    for over in (dict(gx=T(X, 0)), dict(gx=T(X, 4, addr=BASE + 4 * STEP + 4)), dict(gw=T([12], 9)), dict(gb=T([12], 1)), dict(gw=T([12], 4)),
                 dict(gb=T([12], 7)), dict(gx=T(X, 5)), dict(gw=T([12], 3))):
        assert gnb(lib, **over) == dc1d.ERR_ALIAS, over


def rec(lib, ws=(None, 0), **over):
    t = dict(x=S(X, 0), gate=S(X, 1), state=T([3, 12], 2), lens=T([3], 3, I32), y=S(X, 4), last=T([3, 12], 5), states=T([3, 1, 12], 6))
    t.update(over)
    return lib.dc1d_gated_recurrence(*[ref(t[k]) for k in ("x", "gate", "state", "lens", "y", "last", "states")], 1, 0, *ws, None)


def recb(lib, ws=(None, 0), **over):
    t = dict(x=S(X, 0), gate=S(X, 1), states=T([3, 1, 12], 2), lens=T([3], 3, I32), g=S(X, 4), g_last=T([3, 12], 5), gx=S(X, 6),
             gg=S(X, 7), gs=T([3, 12], 8))
    t.update(over)
    return lib.dc1d_gated_recurrence_backward(*[ref(t[k]) for k in ("x", "gate", "states", "lens", "g", "g_last", "gx", "gg", "gs")], 0, 1,
                                              *ws, None)


LARGE = ([3, 10, 0], [3, 10, (1 << 24) + 1], [BIG, 10, 12], [3, (1 << 29) + 1, 1], [-1, 10, 12], [3, -1, 12], [1 << 31, 1, 1],
         [1 << 16, 1 << 15, 1], [1 << 20, 1, 1 << 11], [3, BIG, BIG])


def test_gated_recurrence(lib):
    if no_device():
        for over in ({}, dict(state=None, lens=None, last=None, states=None), dict(y=S(X, 0)), dict(last=T([3, 12], 2)),
                     dict(gate=S(X, 1, stride=(0, 12, 1))), dict(gate=S(X, 1, stride=(0, 0, 1))),
                     dict(x=S(X, 0, stride=(240, 24, 1)), gate=S(X, 0, stride=(240, 24, 1), addr=BASE + 48)),
                     dict(y=S(X, 0, stride=(240, 24, 1), addr=BASE + 48), x=S(X, 0, stride=(240, 24, 1))),
                     dict(x=S([3, 10, 1], 0, stride=(10, 1, 7)), gate=S([3, 10, 1], 1), y=S([3, 10, 1], 4), state=None, last=None,
                          states=None)):
            assert rec(lib, **over) == dc1d.ERR_DEVICE, over
    for k in ("x", "gate", "y"):
        assert rec(lib, **{k: None}) == dc1d.ERR_NULL_PTR
        assert rec(lib, **{k: S(X, 0, addr=0)}) == dc1d.ERR_NULL_PTR
    for k, shape in (("state", [3, 12]), ("last", [3, 12]), ("states", [3, 1, 12])):
        assert rec(lib, **{k: T(shape, 0, addr=0)}) == dc1d.ERR_NULL_PTR
    for over in (dict(x=S(X, 0, 5)), dict(x=S(X, 0, I32)), dict(gate=S(X, 1, BF16)), dict(y=S(X, 4, BF16)), dict(state=T([3, 12], 2, BF16)),
                 dict(states=T([3, 1, 12], 6, I32)), dict(lens=T([3], 3, F32))):
        assert rec(lib, **over) == dc1d.ERR_BAD_DTYPE
    for shape in LARGE:
        assert rec(lib, x=S(shape, 0)) == dc1d.ERR_BAD_SHAPE, shape
    for over in (dict(x=S(X, 0, ndim=4)), dict(x=S(X, 0, ndim=2)), dict(gate=S([3, 10, 13], 1)), dict(y=S([3, 11, 12], 4)),
                 dict(state=T([12], 2)), dict(last=T([3, 13], 5)), dict(states=T([3, 2, 12], 6)), dict(lens=T([10], 3, I32)),
                 dict(x=S(X, 0, stride=(120, 12, 2))), dict(gate=S(X, 1, stride=(120, -12, 1))), dict(gate=S(X, 1, stride=(BIG, 12, 1)))):
        assert rec(lib, **over) == dc1d.ERR_BAD_SHAPE, over
    for over in (dict(y=S(X, 1)), dict(y=S(X, 0, addr=BASE + 4)), dict(y=S(X, 4, stride=(0, 12, 1))), dict(y=S(X, 4, stride=(120, 11, 1))),
                 dict(y=S(X, 2)), dict(last=T([3, 12], 2, addr=BASE + 2 * STEP + 16)), dict(last=T([3, 12], 6)), dict(states=T([3, 1, 12], 2)),
                 dict(states=T([3, 1, 12], 0)), dict(last=T([3, 12], 4)), dict(last=T([3, 12], 3)), dict(y=S(X, 3)),
                 dict(y=S(X, 0, stride=(240, 24, 1)))):
        assert rec(lib, **over) == dc1d.ERR_ALIAS, over
    n = ctypes.c_size_t()
    for f in (lib.dc1d_gated_recurrence_workspace_bytes, lib.dc1d_gated_recurrence_backward_workspace_bytes):
        assert f(ref(S(X, 0)), None) == dc1d.ERR_NULL_PTR and f(None, ctypes.byref(n)) == dc1d.ERR_NULL_PTR
        assert f(ref(S(X, 0, ndim=4)), ctypes.byref(n)) == dc1d.ERR_BAD_SHAPE


def test_gated_recurrence_backward(lib):
    if no_device():
        for over in ({}, dict(lens=None, g_last=None, gx=None, gg=None), dict(gx=S(X, 4)), dict(gs=T([3, 12], 5)), dict(gs=None),
                     dict(gx=S(X, 6, stride=(240, 24, 1)), gg=S(X, 6, stride=(240, 24, 1), addr=BASE + 6 * STEP + 48))):
            assert recb(lib, **over) == dc1d.ERR_DEVICE, over
    for k in ("x", "gate", "g", "states"):
        assert recb(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    for over in (dict(g=S(X, 4, BF16)), dict(gx=S(X, 6, BF16)), dict(gs=T([3, 12], 8, BF16)), dict(states=T([3, 1, 12], 2, BF16))):
        assert recb(lib, **over) == dc1d.ERR_BAD_DTYPE
    for shape in LARGE:
        assert recb(lib, x=S(shape, 0)) == dc1d.ERR_BAD_SHAPE, shape
    for over in (dict(states=T([3, 2, 12], 2)), dict(g=S([3, 10, 11], 4)), dict(gg=S([2, 10, 12], 7)), dict(gs=T([3, 11], 8)),
                 dict(gx=S(X, 6, ndim=4)), dict(lens=T([4], 3, I32))):
        assert recb(lib, **over) == dc1d.ERR_BAD_SHAPE, over
    for over in (dict(gx=S(X, 0)), dict(gg=S(X, 4)), dict(gg=S(X, 6)), dict(gx=S(X, 6, stride=(120, 0, 1))), dict(gs=T([3, 12], 2)),
                 dict(gs=T([3, 12], 6)), dict(gs=T([3, 12], 5, addr=BASE + 5 * STEP + 8)), dict(gx=S(X, 2)), dict(gg=S(X, 3)), dict(gx=S(X, 5)),
                 dict(gs=T([3, 12], 3))):
        assert recb(lib, **over) == dc1d.ERR_ALIAS, over


def test_python_arguments():
    x = torch.zeros(2, 5, 8)
    with pytest.raises(ValueError, match="GPU"):
        sequence.group_norm(x, 2)
    with pytest.raises(ValueError, match="activation"):
        sequence.group_norm(x, 2, activation="gelu")
    with pytest.raises(ValueError, match="activation"):
        sequence.group_norm_backward(x, 2, x, x, x, activation=["silu"])
    with pytest.raises(ValueError, match="GPU"):
        sequence.gated_recurrence(x, x)
    with pytest.raises(ValueError, match="GPU"):
        sequence.gated_recurrence_backward(x, x, x, x)
