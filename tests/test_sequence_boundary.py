"""Host-side checks of the sequence operators' C ABI (no GPU needed): every
malformed call is rejected with the documented status before any device
work.  Data pointers are fake: host validation never dereferences them, and
calls that pass every check are made only where no device is visible."""
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
            "dc1d_layer_norm": [p] * 6 + [f64, p],
            "dc1d_layer_norm_backward_workspace_bytes": [p, i32, p],
            "dc1d_layer_norm_backward": [p] * 8 + [p, n, p],
            "dc1d_rotary": [p] * 8 + [ctypes.c_int32, i32, i32, p],
            "dc1d_attention_workspace_bytes": [p] * 4,
            "dc1d_attention_plan": [p] * 6,
            "dc1d_attention": [p] * 7 + [i32, i64, f64, p, n, p],
            "dc1d_attention_backward_workspace_bytes": [p] * 4,
            "dc1d_attention_backward": [p] * 11 + [i32, i64, f64, p, n, p]}.items():
        getattr(lib, name).argtypes = args
    return lib


def T(shape, slot, dtype=F32, addr=None):
    d = dc1d._Tensor()
    d.data = BASE + slot * STEP if addr is None else (addr or None)
    d.dtype, d.ndim = dtype, len(shape)
    d.shape[:min(len(shape), 4)] = shape[:4]
    return d


def S(shape, slot, dtype=F32, stride=None, addr=None):
    d = Strided()
    d.data = BASE + slot * STEP if addr is None else (addr or None)
    d.dtype, d.ndim = dtype, 4
    if stride is None:
        stride, n = [0] * 4, 1
        for i in (3, 2, 1, 0):
            stride[i] = n
            n *= max(shape[i], 1)
    d.shape[:], d.stride[:] = shape, stride
    return d


def ref(t):
    return None if t is None else ctypes.byref(t)


def reaches_device(status):
    return status == dc1d.ERR_DEVICE


def no_device():
    return torch.cuda.device_count() == 0


def ln(lib, eps=1e-5, **over):
    t = dict(x=T([2, 8, 20], 0), w=T([8], 1), b=T([8], 2), y=T([2, 8, 20], 3), mean=T([2, 20], 4), rstd=T([2, 20], 5))
    t.update(over)
    return lib.dc1d_layer_norm(*[ref(t[k]) for k in ("x", "w", "b", "y", "mean", "rstd")], eps, None)


def test_layer_norm(lib):
    if no_device():
        assert reaches_device(ln(lib))
        assert reaches_device(ln(lib, w=None, b=None, mean=None, rstd=None))
        assert reaches_device(ln(lib, y=T([2, 8, 20], 0)))  # in place
        assert reaches_device(ln(lib, x=T([3, 8], 0), y=T([3, 8], 3), mean=T([3], 4), rstd=T([3], 5)))
        assert reaches_device(ln(lib, x=T([1, 8, 4, 5], 0), y=T([1, 8, 4, 5], 3), mean=T([1, 4, 5], 4), rstd=T([1, 4, 5], 5)))
    for k in ("x", "y"):
        assert ln(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    assert ln(lib, w=T([8], 1, addr=0)) == dc1d.ERR_NULL_PTR
    assert ln(lib, x=T([2, 8, 20], 0, 7)) == dc1d.ERR_BAD_DTYPE
    assert ln(lib, x=T([2, 8, 20], 0, I32)) == dc1d.ERR_BAD_DTYPE
    assert ln(lib, w=T([8], 1, BF16)) == dc1d.ERR_BAD_DTYPE
    assert ln(lib, mean=T([2, 20], 4, BF16)) == dc1d.ERR_BAD_DTYPE
    for shape in ([8], [2, 0, 20], [2, (1 << 24) + 1, 20], [BIG, 8, 20], [2, 8, BIG], [-1, 8, 20], [2, 8, -1], [1 << 31, 8, 1],
                  [1 << 16, 1, 1 << 15], [BIG, 8, BIG, BIG]):
        assert ln(lib, x=T(shape, 0)) == dc1d.ERR_BAD_SHAPE, shape
    assert ln(lib, y=T([2, 8, 21], 3)) == dc1d.ERR_BAD_SHAPE
    assert ln(lib, b=T([9], 2)) == dc1d.ERR_BAD_SHAPE
    assert ln(lib, rstd=T([2, 8], 5)) == dc1d.ERR_BAD_SHAPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert ln(lib, eps) == dc1d.ERR_BAD_ARG
    assert ln(lib, y=T([2, 8, 20], 0, addr=BASE + 4)) == dc1d.ERR_ALIAS
    assert ln(lib, y=T([2, 8, 20], 1)) == dc1d.ERR_ALIAS
    assert ln(lib, mean=T([2, 20], 5)) == dc1d.ERR_ALIAS
    assert ln(lib, rstd=T([2, 20], 0)) == dc1d.ERR_ALIAS


def lnb(lib, ws=(None, 0), **over):
    t = dict(x=T([2, 8, 20], 0), w=T([8], 1), g=T([2, 8, 20], 2), mean=T([2, 20], 3), rstd=T([2, 20], 4),
             gx=T([2, 8, 20], 5), gw=T([8], 6), gb=T([8], 7))
    t.update(over)
    return lib.dc1d_layer_norm_backward(*[ref(t[k]) for k in ("x", "w", "g", "mean", "rstd", "gx", "gw", "gb")], *ws, None)


def test_layer_norm_backward(lib):
    if no_device():
        assert reaches_device(lnb(lib))
        assert reaches_device(lnb(lib, gx=T([2, 8, 20], 2)))  # over the output's gradient
    for k in ("x", "g", "mean", "rstd"):
        assert lnb(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    assert lnb(lib, g=T([2, 8, 20], 2, BF16)) == dc1d.ERR_BAD_DTYPE
    assert lnb(lib, gw=T([8], 6, BF16)) == dc1d.ERR_BAD_DTYPE
    assert lnb(lib, gx=T([2, 8, 19], 5)) == dc1d.ERR_BAD_SHAPE
    assert lnb(lib, gb=T([7], 7)) == dc1d.ERR_BAD_SHAPE
    assert lnb(lib, gx=T([2, 8, 20], 0)) == dc1d.ERR_ALIAS
    assert lnb(lib, gw=T([8], 7)) == dc1d.ERR_ALIAS
    n = ctypes.c_size_t()
    assert lib.dc1d_layer_norm_backward_workspace_bytes(ref(T([8], 0)), 1, ctypes.byref(n)) == dc1d.ERR_BAD_SHAPE
    assert lib.dc1d_layer_norm_backward_workspace_bytes(ref(T([8, 8], 0)), 1, None) == dc1d.ERR_NULL_PTR


def rot(lib, sections=(12, 20), axes=None, **over):
    t = dict(q=S([2, 5, 4, 64], 0), k=S([2, 5, 2, 64], 1), cos=T([9, 32], 2), sin=T([9, 32], 3), pos=T([2, 5, 2], 4, I32),
             qo=S([2, 5, 4, 64], 5), ko=S([2, 5, 2, 64], 6))
    t.update(over)
    n = len(sections) if axes is None else axes
    return lib.dc1d_rotary(*[ref(t[k]) for k in ("q", "k", "cos", "sin", "pos", "qo", "ko")],
                           (ctypes.c_int64 * 8)(*sections), n, 0, 0, None)


def test_rotary(lib):
    row = [5 * 8 * 64, 8 * 64, 64, 1]
    if no_device():
        assert reaches_device(rot(lib))
        assert reaches_device(rot(lib, k=None, ko=None))
        assert reaches_device(rot(lib, pos=T([1, 5, 2], 4, I32)))
        assert reaches_device(rot(lib, qo=S([2, 5, 4, 64], 0), ko=S([2, 5, 2, 64], 1)))  # in place
        # in place on head slices of one buffer
        q, k = S([2, 5, 4, 64], 0, stride=row), S([2, 5, 2, 64], 0, stride=row, addr=BASE + 4 * 64 * 4)
        assert reaches_device(rot(lib, q=q, k=k, qo=q, ko=k))
    for k in ("q", "cos", "sin", "pos", "qo", "ko", "k"):
        assert rot(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    for sections in ((), (12, 20, 1), (33,), (-1, 33), (0, 0), (BIG, BIG)):
        assert rot(lib, sections) == dc1d.ERR_BAD_ARG, sections
    assert rot(lib, (8, 8, 8, 8, 0), 5) == dc1d.ERR_BAD_ARG
    assert rot(lib, (12, 19)) == dc1d.ERR_BAD_SHAPE  # the tables hold 32 pairs
    assert rot(lib, (32,)) == dc1d.ERR_BAD_SHAPE     # positions have two axes
    assert rot(lib, pos=T([2, 5, 2], 4)) == dc1d.ERR_BAD_DTYPE
    assert rot(lib, cos=T([9, 32], 2, BF16)) == dc1d.ERR_BAD_DTYPE
    assert rot(lib, ko=S([2, 5, 2, 64], 6, BF16)) == dc1d.ERR_BAD_DTYPE
    assert rot(lib, sin=T([8, 32], 3)) == dc1d.ERR_BAD_SHAPE
    assert rot(lib, k=S([2, 4, 2, 64], 1), ko=S([2, 4, 2, 64], 6)) == dc1d.ERR_BAD_SHAPE
    assert rot(lib, q=S([2, 5, 4, 64], 0, stride=[1280, 256, 64, 2])) == dc1d.ERR_BAD_SHAPE
    assert rot(lib, q=S([2, 5, 4, 64], 0, stride=[-1, 256, 64, 1])) == dc1d.ERR_BAD_SHAPE
    assert rot(lib, q=S([BIG, BIG, 4, 64], 0, stride=[1] * 4)) == dc1d.ERR_BAD_SHAPE
    assert rot(lib, qo=S([2, 5, 4, 64], 5, stride=[0, 256, 64, 1])) == dc1d.ERR_ALIAS
    assert rot(lib, qo=S([2, 5, 4, 64], 5, stride=[1280, 255, 64, 1])) == dc1d.ERR_ALIAS
    assert rot(lib, qo=S([2, 5, 4, 64], 1)) == dc1d.ERR_ALIAS   # on the other input
    assert rot(lib, qo=S([2, 5, 4, 64], 0, addr=BASE + 256)) == dc1d.ERR_ALIAS
    assert rot(lib, qo=S([2, 5, 4, 64], 2)) == dc1d.ERR_ALIAS   # on the tables
    # slices of one buffer that share a head
    q, k = S([2, 5, 4, 64], 0, stride=row), S([2, 5, 2, 64], 0, stride=row, addr=BASE + 3 * 64 * 4)
    assert rot(lib, q=q, k=k, qo=q, ko=k) == dc1d.ERR_ALIAS


def att(lib, causal=0, window=0, scale=0.125, ws=(None, 0), **over):
    t = dict(q=S([2, 5, 4, 64], 0), k=S([2, 7, 2, 64], 1), v=S([2, 7, 2, 64], 2), lens=T([2], 3, I32), start=T([2], 4, I32),
             out=S([2, 5, 4, 64], 5), lse=T([2, 4, 5], 6))
    t.update(over)
    return lib.dc1d_attention(*[ref(t[k]) for k in ("q", "k", "v", "lens", "start", "out", "lse")], causal, window, scale,
                              *ws, None)


def test_attention(lib):
    if no_device():
        assert reaches_device(att(lib))
        assert reaches_device(att(lib, 1, BIG, lens=None, start=None, lse=None))
        assert reaches_device(att(lib, k=S([2, 7, 2, 64], 1, stride=[0, 64, 0, 1])))  # a repeated input
        assert reaches_device(att(lib, k=S([2, 0, 2, 64], 1, addr=0), v=S([2, 0, 2, 64], 2, addr=0)))
    for k in ("q", "k", "v", "out"):
        assert att(lib, **{k: None}) == dc1d.ERR_NULL_PTR
        shape = [2, 5, 4, 64] if k in ("q", "out") else [2, 7, 2, 64]
        assert att(lib, **{k: S(shape, 0, addr=0)}) == dc1d.ERR_NULL_PTR
    assert att(lib, lens=T([2], 3, I32, addr=0)) == dc1d.ERR_NULL_PTR
    assert att(lib, q=S([2, 5, 4, 64], 0, I32)) == dc1d.ERR_BAD_DTYPE
    assert att(lib, v=S([2, 7, 2, 64], 2, BF16)) == dc1d.ERR_BAD_DTYPE
    assert att(lib, out=S([2, 5, 4, 64], 5, BF16)) == dc1d.ERR_BAD_DTYPE
    assert att(lib, start=T([2], 4)) == dc1d.ERR_BAD_DTYPE
    assert att(lib, lse=T([2, 4, 5], 6, BF16)) == dc1d.ERR_BAD_DTYPE
    for shape in ([2, 7, 3, 64], [3, 7, 2, 64], [2, 7, 2, 32], [2, 7, 0, 64], [2, (1 << 29) + 1, 2, 64], [BIG, 7, 2, 64],
                  [2, BIG, BIG, 64], [2, -7, 2, 64]):
        stride = [1] * 4
        assert att(lib, k=S(shape, 1, stride=stride), v=S(shape, 2, stride=stride)) == dc1d.ERR_BAD_SHAPE, shape
    assert att(lib, v=S([2, 6, 2, 64], 2)) == dc1d.ERR_BAD_SHAPE
    assert att(lib, out=S([2, 5, 2, 64], 5)) == dc1d.ERR_BAD_SHAPE
    assert att(lib, lse=T([2, 5, 4], 6)) == dc1d.ERR_BAD_SHAPE
    assert att(lib, lens=T([3], 3, I32)) == dc1d.ERR_BAD_SHAPE
    assert att(lib, k=S([2, 7, 2, 64], 1, stride=[BIG, 128, 64, 1])) == dc1d.ERR_BAD_SHAPE
    big = [S([1, 5, 1, 129], i) for i in (0, 1, 2, 5)]
    assert att(lib, q=big[0], k=big[1], v=big[2], out=big[3], lens=None, start=None, lse=None) == dc1d.ERR_BAD_SHAPE
    many = [S([1 << 24, 1, 1, 1], i) for i in (0, 1, 2, 5)]
    assert att(lib, q=many[0], k=many[1], v=many[2], out=many[3], lens=None, start=None, lse=None) == dc1d.ERR_BAD_SHAPE
    assert att(lib, window=-1) == dc1d.ERR_BAD_ARG
    for scale in (0.0, -0.1, float("nan"), float("inf"), 1e-60):
        assert att(lib, scale=scale) == dc1d.ERR_BAD_ARG
    for slot in (0, 1, 2, 3, 4, 6):
        assert att(lib, out=S([2, 5, 4, 64], slot)) == dc1d.ERR_ALIAS
    assert att(lib, lse=T([2, 4, 5], 1)) == dc1d.ERR_ALIAS
    assert att(lib, out=S([2, 5, 4, 64], 5, stride=[1280, 256, 32, 1])) == dc1d.ERR_ALIAS


def attb(lib, **over):
    t = dict(q=S([2, 5, 4, 64], 0), k=S([2, 7, 2, 64], 1), v=S([2, 7, 2, 64], 2), lens=T([2], 3, I32), start=None,
             out=S([2, 5, 4, 64], 5), lse=T([2, 4, 5], 6), g=S([2, 5, 4, 64], 7), gq=S([2, 5, 4, 64], 8),
             gk=S([2, 7, 2, 64], 9), gv=S([2, 7, 2, 64], 10))
    t.update(over)
    return lib.dc1d_attention_backward(*[ref(t[k]) for k in ("q", "k", "v", "lens", "start", "out", "lse", "g", "gq", "gk", "gv")],
                                       0, 0, 0.125, None, 0, None)


def test_attention_backward(lib):
    if no_device():
        assert reaches_device(attb(lib))
        assert reaches_device(attb(lib, gq=None, gk=None))
        # gradients as head slices of one buffer
        row = [7 * 256, 256, 64, 1]
        assert reaches_device(attb(lib, gk=S([2, 7, 2, 64], 9, stride=row), gv=S([2, 7, 2, 64], 9, stride=row, addr=BASE + 9 * STEP + 512)))
    for k in ("q", "k", "v", "out", "lse", "g"):
        assert attb(lib, **{k: None}) == dc1d.ERR_NULL_PTR
    assert attb(lib, g=S([2, 5, 4, 64], 7, BF16)) == dc1d.ERR_BAD_DTYPE
    assert attb(lib, gk=S([2, 5, 4, 64], 9)) == dc1d.ERR_BAD_SHAPE
    assert attb(lib, gq=S([2, 7, 2, 64], 8)) == dc1d.ERR_BAD_SHAPE
    assert attb(lib, gv=S([2, 7, 2, 64], 9)) == dc1d.ERR_ALIAS
    for slot in (0, 1, 2, 3, 5, 6, 7):
        assert attb(lib, gq=S([2, 5, 4, 64], slot)) == dc1d.ERR_ALIAS
    row = [7 * 256, 256, 64, 1]
    assert attb(lib, gk=S([2, 7, 2, 64], 9, stride=row), gv=S([2, 7, 2, 64], 9, stride=row, addr=BASE + 9 * STEP + 508)) == dc1d.ERR_ALIAS
    n = ctypes.c_size_t()
    q, k = S([2, 5, 4, 64], 0), S([2, 7, 3, 64], 1)
    assert lib.dc1d_attention_workspace_bytes(ref(q), ref(k), ref(k), ctypes.byref(n)) == dc1d.ERR_BAD_SHAPE
    assert lib.dc1d_attention_backward_workspace_bytes(ref(q), ref(k), ref(k), ctypes.byref(n)) == dc1d.ERR_BAD_SHAPE
    assert lib.dc1d_attention_plan(ref(q), ref(k), ref(k), None, None, None) == dc1d.ERR_BAD_SHAPE


def test_python_refusals():
    x = torch.zeros(2, 8)
    for fn in (lambda: sequence.layer_norm(x), lambda: sequence.attention(*[torch.zeros(1, 2, 2, 8)] * 3),
               lambda: sequence.rotary(torch.zeros(1, 2, 2, 8), None, x, x, x, (4,))):
        with pytest.raises(ValueError):  # tensors on the host
            fn()
