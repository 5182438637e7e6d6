"""Binding over libdc1d's sequence operators (include/dc1d.h): layer norm over
axis 1, rotary positions with several axes, and attention, each with its
gradient.

Argument marshalling only, like ``dc1d``: torch tensors become descriptors,
the work is enqueued on torch's current stream, status codes become
exceptions, and there is no fallback of any kind.  Small calls are bound by
the host, so the marshalling is compiled (csrc/bind_seq.cpp, built in-tree as
``_seq.so``).
"""
from __future__ import annotations

import ctypes

import torch

from . import dc1d
from .dc1d import _check, _nullctx, _workspace

_ENTRIES = ("dc1d_layer_norm", "dc1d_layer_norm_backward_workspace_bytes", "dc1d_layer_norm_backward", "dc1d_rotary",
            "dc1d_attention_workspace_bytes", "dc1d_attention", "dc1d_attention_backward_workspace_bytes",
            "dc1d_attention_backward")

_bound = None


def _binding():
    """The compiled binding, given the library's entries."""
    global _bound
    if _bound is None:
        lib = dc1d.load_library()
        try:
            from . import _seq
        except ImportError as e:
            raise ImportError("_seq.so is not built; run __graft_entry__.build()") from e
        _seq.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in _ENTRIES))
        _bound = _seq
    return _bound


_here = _nullctx()


def _on(index):
    """torch.cuda.device(index), or nothing when it is already current (or no
    device, which the binding refuses)."""
    return _here if index < 0 or index == torch.cuda.current_device() else torch.cuda.device(index)


def _stream(index):
    return torch._C._cuda_getCurrentRawStream(index) if index >= 0 else 0


def _get(nbytes, index):
    return _workspace(nbytes, torch.device("cuda", index))


def layer_norm(x, weight=None, bias=None, eps=1e-5, with_stats=False, out=None):
    """Layer norm over axis 1 of x [N, C], [B, C, L] or [B, C, H, W] (float32
    or bfloat16, contiguous): (x - mean) / sqrt(var + eps) * weight + bias.
    Returns y (allocated unless given as ``out``, which may be x), or with
    with_stats (y, mean, rstd), float32 tensors of x's shape without axis 1."""
    seq = _bound or _binding()
    index = x.get_device()
    with _on(index):
        status, y, mean, rstd = seq.layer_norm(x, weight, bias, eps, with_stats, out, _stream(index))
    if status:
        _check(status, "dc1d_layer_norm")
    return (y, mean, rstd) if with_stats else y


def layer_norm_backward(x, grad_out, mean, rstd, weight=None, need=("x", "weight", "bias"), workspace=None):
    """Gradients of sum(grad_out * layer_norm(x, weight, bias)) from the
    forward's mean and rstd: a dict with the requested keys, each gradient in
    x's dtype."""
    seq = _bound or _binding()
    index = x.get_device()
    with _on(index):
        status, *grads = seq.layer_norm_backward(x, grad_out, mean, rstd, weight, "x" in need, "weight" in need, "bias" in need,
                                                 workspace, _get, _stream(index))
    if status:
        _check(status, "dc1d_layer_norm_backward")
    return {n: g for n, g in zip(("x", "weight", "bias"), grads) if g is not None}


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
    seq = _bound or _binding()
    index = q.get_device()
    q_out, k_out = out if out is not None else (None, None)
    with _on(index):
        status, q_out, k_out = seq.rotary(q, k, cos, sin, positions, tuple(sections), interleaved, inverse, q_out, k_out,
                                          _stream(index))
    if status:
        _check(status, "dc1d_rotary")
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
    seq = _bound or _binding()
    index = q.get_device()
    with _on(index):
        status, out, lse = seq.attention(q, k, v, causal, window, _scale(scale, q), kv_lens, q_start, with_lse, out, workspace,
                                         _get, _stream(index))
    if status:
        _check(status, "dc1d_attention")
    return (out, lse) if with_lse else out


def attention_plan(q, k, v) -> dict:
    """Which kernel an attention call with these tensors uses, its workgroups
    and into how many parts the keys are split."""
    lib = dc1d.load_library()
    name, grid, splits = ctypes.c_char_p(), ctypes.c_int64(), ctypes.c_int32()
    with _on(q.get_device()):
        _check(lib.dc1d_attention_plan(*(ctypes.byref(_strided(t)) for t in (q, k, v)), ctypes.byref(name),
                                       ctypes.byref(grid), ctypes.byref(splits)), "dc1d_attention_plan")
    return {"kernel": name.value.decode(), "grid": grid.value, "splits": splits.value}


def attention_backward(q, k, v, out, lse, grad_out, causal=False, window=0, scale=None, kv_lens=None, q_start=None,
                       need=("q", "k", "v"), grads=None, workspace=None):
    """Gradients of sum(grad_out * attention(q, k, v, ...)) from the forward's
    inputs, out and lse: a dict with the requested keys, each shaped like its
    input (allocated, or given in ``grads`` under its key: any strides, for
    instance head slices of one buffer)."""
    seq = _bound or _binding()
    index = q.get_device()
    given = grads or {}
    want = [(given.get(n) if given.get(n) is not None else True) if n in need else None for n in "qkv"]
    with _on(index):
        status, *got = seq.attention_backward(q, k, v, out, lse, grad_out, causal, window, _scale(scale, q), kv_lens, q_start,
                                              *want, workspace, _get, _stream(index))
    if status:
        _check(status, "dc1d_attention_backward")
    return {n: g for n, g in zip("qkv", got) if g is not None}


def _scale(scale, q):
    return q.shape[-1] ** -0.5 if scale is None and q.dim() and q.shape[-1] else 1.0 if scale is None else scale


class _Strided(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4), ("stride", ctypes.c_int64 * 4)]


def _strided(t):
    d = _Strided()
    d.data, d.dtype, d.ndim = t.data_ptr(), dc1d._DTYPES.get(t.dtype, -1), t.dim()
    d.shape[:min(d.ndim, 4)] = t.shape[:4]
    d.stride[:min(d.ndim, 4)] = t.stride()[:4]
    return d
