"""ctypes binding over libdc1d's sequence operators (include/dc1d.h): layer
norm over axis 1, rotary positions with several axes, and attention, each
with its gradient.

Argument marshalling only, like ``dc1d``: torch tensors become descriptors,
the work is enqueued on torch's current stream, status codes become
exceptions, and there is no fallback of any kind.
"""
from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import dc1d
from .dc1d import _check, _contig, _nullctx, _workspace

DC1D_I32 = 2
_DTYPES = {torch.float32: dc1d.DC1D_F32, torch.bfloat16: dc1d.DC1D_BF16, torch.int32: DC1D_I32}

# Descriptors are packed bytes in the layout of the C structures (small calls
# are bound by the host; filling ctypes structures takes several times as
# long): dc1d_tensor by rank, the unused shape entries zero, and dc1d_strided.
_TENSOR = [struct.Struct("Pii%dq%dx" % (n, 8 * (4 - n))).pack for n in range(5)]
_STRIDED = struct.Struct("Pii8q").pack

_declared = None


def _library():
    global _declared
    if _declared is None:
        lib = dc1d.load_library()
        p, n, i32, i64, f64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_int64, ctypes.c_double
        for name, args in {
                "dc1d_layer_norm": [p] * 6 + [f64, p],
                "dc1d_layer_norm_backward_workspace_bytes": [p, i32, p],
                "dc1d_layer_norm_backward": [p] * 8 + [p, n, p],
                "dc1d_rotary": [p] * 8 + [ctypes.c_int32, i32, i32, p],
                "dc1d_attention_workspace_bytes": [p] * 3 + [p],
                "dc1d_attention_plan": [p] * 3 + [p] * 3,
                "dc1d_attention": [p] * 7 + [i32, i64, f64, p, n, p],
                "dc1d_attention_backward_workspace_bytes": [p] * 3 + [p],
                "dc1d_attention_backward": [p] * 11 + [i32, i64, f64, p, n, p]}.items():
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            fn.argtypes = args
        _declared = lib
    return _declared


def _desc(t, name):
    """A contiguous tensor's descriptor."""
    if t is None:
        return None
    if not t.is_contiguous():
        _contig(t, name)
    shape = t.shape
    n = len(shape)
    if n > 4:  # the rank alone decides: refused
        return _TENSOR[4](t.data_ptr(), _DTYPES.get(t.dtype, -1), n, *shape[:4])
    return _TENSOR[n](t.data_ptr(), _DTYPES.get(t.dtype, -1), n, *shape)


def _strided(t, name):
    """A tensor of rank 4 with its strides."""
    if t is None:
        return None
    if t.dim() != 4:
        raise ValueError("%s must have four dimensions" % name)
    return _STRIDED(t.data_ptr(), _DTYPES.get(t.dtype, -1), 4, *t.shape, *t.stride())


def _device_of(first, *rest):
    """The index of the GPU that all the tensors (or Nones) are on."""
    index = first.get_device()
    if index < 0:
        raise ValueError("tensors must be on the GPU")
    for t in rest:
        if t is not None and t.get_device() != index:
            raise ValueError("all tensors must be on one device")
    return index


_here = _nullctx()


def _on(index):
    return _here if index == torch.cuda.current_device() else torch.cuda.device(index)


def _stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _sized(query, *args):
    n = ctypes.c_size_t(0)
    _check(query(*args, ctypes.byref(n)), query.__name__)
    return n.value


def _scratch(nbytes, workspace, device):
    """(pointer, bytes) of the caller's workspace or of this stream's cached one."""
    if workspace is None:
        if nbytes == 0:
            return None, 0
        workspace = _workspace(nbytes, device)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def layer_norm(x, weight=None, bias=None, eps=1e-5, with_stats=False, out=None):
    """Layer norm over axis 1 of x [N, C], [B, C, L] or [B, C, H, W] (float32
    or bfloat16, contiguous): (x - mean) / sqrt(var + eps) * weight + bias.
    Returns y (allocated unless given as ``out``, which may be x), or with
    with_stats (y, mean, rstd), float32 tensors of x's shape without axis 1."""
    lib = _library()
    index = _device_of(x, weight, bias, out)
    y = torch.empty_like(x) if out is None else out
    mean = rstd = None
    if with_stats:
        mean = x.new_empty(x.shape[:1] + x.shape[2:], dtype=torch.float32)
        rstd = torch.empty_like(mean)
    d = (_desc(x, "x"), _desc(weight, "weight"), _desc(bias, "bias"), _desc(y, "out"), _desc(mean, "mean"),
         _desc(rstd, "rstd"))
    with _on(index):
        _check(lib.dc1d_layer_norm(*d, eps, _stream(index)), "dc1d_layer_norm")
    return (y, mean, rstd) if with_stats else y


def layer_norm_backward(x, grad_out, mean, rstd, weight=None, need=("x", "weight", "bias"), workspace=None):
    """Gradients of sum(grad_out * layer_norm(x, weight, bias)) from the
    forward's mean and rstd: a dict with the requested keys, each gradient in
    x's dtype."""
    lib = _library()
    index = _device_of(x, grad_out, mean, rstd, weight)
    grads = {k: torch.empty_like(x) if k == "x" else x.new_empty(x.shape[1]) for k in need}
    gx, gw, gb = (grads.get(k) for k in ("x", "weight", "bias"))
    d = (_desc(x, "x"), _desc(weight, "weight"), _desc(grad_out, "grad_out"), _desc(mean, "mean"), _desc(rstd, "rstd"),
         _desc(gx, "grad_x"), _desc(gw, "grad_weight"), _desc(gb, "grad_bias"))
    with _on(index):
        params = int(gw is not None or gb is not None)
        nbytes = _sized(lib.dc1d_layer_norm_backward_workspace_bytes, d[0], params) if params else 0
        _check(lib.dc1d_layer_norm_backward(*d, *_scratch(nbytes, workspace, x.device), _stream(index)),
               "dc1d_layer_norm_backward")
    return grads


def rotary(q, k, cos, sin, positions, sections, interleaved=False, inverse=False, out=None):
    """Rotary positions of q [B, L, Hq, D] and k [B, L, Hkv, D] (or None):
    pair i turns by the tables' (cos, sin [P, R], float32) angle of position
    positions[b, l, axis] (int32 [B, L, A], or [1, L, A] shared), the axis
    being the section that i falls in (``sections``: pairs per axis, adding
    up to R).  A pair is elements (i, R + i), or (2i, 2i + 1) if interleaved;
    elements past 2 R are copied.  inverse=True turns back: the gradient's
    rotation.  q and k may have any strides over a contiguous last dimension.
    Returns the pair (q', k'), allocated unless given as ``out`` = (q', k'),
    which may be (q, k)."""
    lib = _library()
    q_out, k_out = out if out is not None else (None, None)
    index = _device_of(q, k, cos, sin, positions, q_out, k_out)
    if q_out is None:
        q_out = q.new_empty(q.shape)
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = k.new_empty(k.shape)
    n = len(sections)
    s = (_strided(q, "q"), _strided(k, "k"), _desc(cos, "cos"), _desc(sin, "sin"), _desc(positions, "positions"),
         _strided(q_out, "out"), _strided(k_out, "out"))
    with _on(index):
        _check(lib.dc1d_rotary(*s, struct.pack("%dq" % n, *sections), n, int(interleaved), int(inverse),
                               _stream(index)), "dc1d_rotary")
    return q_out, k_out


def attention(q, k, v, causal=False, window=0, scale=None, kv_lens=None, q_start=None, with_lse=False, out=None,
              workspace=None):
    """Attention of q [B, Lq, Hq, D] over k, v [B, Lk, Hkv, D] (Hkv dividing
    Hq, D <= 128; any strides over a contiguous last dimension).  Query i of
    batch b stands at p = q_start[b] + i (int32 [B]; None: Lk - Lq + i) and
    sees the keys j < kv_lens[b] (int32 [B]; None: Lk) with j <= p if causal
    and |p - j| < window if window > 0; one that sees none gives 0 (and lse
    -inf).  scale defaults to 1 / sqrt(D).  Returns out (allocated unless
    given), or with with_lse (out, lse), lse float32 [B, Hq, Lq]."""
    lib = _library()
    index = _device_of(q, k, v, kv_lens, q_start, out)
    s = (_strided(q, "q"), _strided(k, "k"), _strided(v, "v"))
    if out is None:
        out = q.new_empty(q.shape)
    B, Lq, Hq, D = q.shape
    lse = q.new_empty((B, Hq, Lq), dtype=torch.float32) if with_lse else None
    more = (_desc(kv_lens, "kv_lens"), _desc(q_start, "q_start"), _strided(out, "out"), _desc(lse, "lse"))
    with _on(index):
        nbytes = _sized(lib.dc1d_attention_workspace_bytes, *s)
        _check(lib.dc1d_attention(*s, *more, int(causal), window, _scale(scale, D),
                                  *_scratch(nbytes, workspace, q.device), _stream(index)), "dc1d_attention")
    return (out, lse) if with_lse else out


def attention_plan(q, k, v) -> dict:
    """Which kernel an attention call with these tensors uses, its workgroups
    and into how many parts the keys are split."""
    lib = _library()
    index = _device_of(q, k, v)
    s = (_strided(q, "q"), _strided(k, "k"), _strided(v, "v"))
    name, grid, splits = ctypes.c_char_p(), ctypes.c_int64(), ctypes.c_int32()
    with _on(index):
        _check(lib.dc1d_attention_plan(*s, ctypes.byref(name), ctypes.byref(grid), ctypes.byref(splits)),
               "dc1d_attention_plan")
    return {"kernel": name.value.decode(), "grid": grid.value, "splits": splits.value}


def attention_backward(q, k, v, out, lse, grad_out, causal=False, window=0, scale=None, kv_lens=None, q_start=None,
                       need=("q", "k", "v"), grads=None, workspace=None):
    """Gradients of sum(grad_out * attention(q, k, v, ...)) from the forward's
    inputs, out and lse: a dict with the requested keys, each shaped like its
    input (allocated, or given in ``grads`` under its key: any strides, for
    instance head slices of one buffer)."""
    lib = _library()
    like = {"q": q, "k": k, "v": v}
    given = grads or {}
    grads = {n: given[n] if given.get(n) is not None else q.new_empty(like[n].shape)
             for n in need}
    index = _device_of(q, k, v, out, lse, grad_out, kv_lens, q_start, *grads.values())
    s = (_strided(q, "q"), _strided(k, "k"), _strided(v, "v"))
    more = (_desc(kv_lens, "kv_lens"), _desc(q_start, "q_start"), _strided(out, "out"), _desc(lse, "lse"),
            _strided(grad_out, "grad_out"), *(_strided(grads.get(n), "grads") for n in ("q", "k", "v")))
    with _on(index):
        nbytes = _sized(lib.dc1d_attention_backward_workspace_bytes, *s)
        _check(lib.dc1d_attention_backward(*s, *more, int(causal), window, _scale(scale, q.shape[3]),
                                           *_scratch(nbytes, workspace, q.device), _stream(index)),
               "dc1d_attention_backward")
    return grads


def _scale(scale, D):
    return 1.0 / math.sqrt(max(D, 1)) if scale is None else float(scale)
