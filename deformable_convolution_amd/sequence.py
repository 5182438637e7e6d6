"""Binding over libdc1d's sequence operators (include/dc1d.h): layer norm over
axis 1, rotary positions with several axes, attention, group norm with an
activation over channels-last positions, and a gated linear recurrence, each
with its gradient.

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
            "dc1d_attention_backward", "dc1d_group_norm_workspace_bytes", "dc1d_group_norm",
            "dc1d_group_norm_backward_workspace_bytes", "dc1d_group_norm_backward", "dc1d_gated_recurrence_workspace_bytes",
            "dc1d_gated_recurrence", "dc1d_gated_recurrence_backward_workspace_bytes", "dc1d_gated_recurrence_backward")

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


_ACTIVATIONS = {None: 0, "relu": 1, "silu": 2}


def _activation(name):
    try:
        return _ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError("activation must be None, 'relu' or 'silu', not %r" % (name,)) from None


def group_norm(x, groups, weight=None, bias=None, eps=1e-5, activation=None, lens=None, with_stats=False, out=None, workspace=None):
    """Group norm of x [N, C], [B, L, C] or [B, H, W, C] (float32 or bfloat16,
    contiguous: channels last) over a sample's positions and each of ``groups``
    runs of C / groups channels: (x - mean) / sqrt(var + eps) * weight + bias,
    then ``activation`` (None, "relu" or "silu").  With lens (int32 [B], for
    [B, L, C]) only the first lens[b] positions count, and the others give 0.
    Returns y (allocated unless given as ``out``, which may be x), or with
    with_stats (y, mean, rstd), float32 [B, groups]."""
    seq = _bound or _binding()
    index = x.get_device()
    with _on(index):
        status, y, mean, rstd = seq.group_norm(x, groups, weight, bias, lens, eps, _activation(activation), with_stats, out, workspace,
                                               _get, _stream(index))
    if status:
        _check(status, "dc1d_group_norm")
    return (y, mean, rstd) if with_stats else y


def group_norm_backward(x, groups, grad_out, mean, rstd, weight=None, bias=None, activation=None, lens=None,
                        need=("x", "weight", "bias"), workspace=None):
    """Gradients of sum(grad_out * group_norm(x, groups, weight, bias, ...)) from
    the forward's mean and rstd: a dict with the requested keys, each gradient
    in x's dtype.  bias is that of the forward (the activation's derivative
    depends on it)."""
    seq = _bound or _binding()
    index = x.get_device()
    with _on(index):
        status, *grads = seq.group_norm_backward(x, groups, grad_out, mean, rstd, weight, bias, lens, _activation(activation),
                                                 "x" in need, "weight" in need, "bias" in need, workspace, _get, _stream(index))
    if status:
        _check(status, "dc1d_group_norm_backward")
    return {n: g for n, g in zip(("x", "weight", "bias"), grads) if g is not None}


def gated_recurrence(x, gate, state=None, lens=None, blend=False, reverse=False, with_states=False, out=None, last=None,
                     workspace=None):
    """The recurrence h_t = a_t h_{t-1} + u_t with a = sigmoid(gate) and u = x, or
    (1 - a) x if blend, along the positions of x [B, L, C] (gate alike; any
    strides over contiguous channels, also 0: ``gate.expand(...)``), from its
    end if reverse.  ``state`` is the state ahead of the first position (float32
    [B, C]; None: zeros); with lens (int32 [B]) a sequence ends after lens[b]
    positions, and those past it give 0.  Returns (y, last): every position's
    state in x's dtype (allocated unless given as ``out``, which may be x), and
    the last one, float32 [B, C] (allocated unless given as ``last``, which may
    be ``state``: a sequence taken up again, a position at a time or more).
    with_states adds the states that the backward pass starts from, float32
    [B, ceil(L / 64), C]."""
    seq = _bound or _binding()
    index = x.get_device()
    with _on(index):
        status, y, last, states = seq.gated_recurrence(x, gate, state, lens, blend, reverse, with_states, out, last, workspace, _get,
                                                       _stream(index))
    if status:
        _check(status, "dc1d_gated_recurrence")
    return (y, last, states) if with_states else (y, last)


def gated_recurrence_backward(x, gate, states, grad_out, grad_last=None, lens=None, blend=False, reverse=False,
                              need=("x", "gate", "state"), grads=None, workspace=None):
    """Gradients of sum(grad_out * y) + sum(grad_last * last) for
    y, last = gated_recurrence(x, gate, ...) from the forward's inputs and states
    (grad_last None: zeros): a dict with the requested keys, x's and gate's of
    x's shape and dtype, state's float32 [B, C] (allocated, or given in
    ``grads`` under its key: for x and gate any strides, for instance slices of
    one buffer).  A gate expanded along a dimension gets the gradient of its
    expanded elements, to be summed along it."""
    seq = _bound or _binding()
    index = x.get_device()
    given = grads or {}
    want = [(given.get(n) if given.get(n) is not None else True) if n in need else None for n in ("x", "gate", "state")]
    with _on(index):
        status, *got = seq.gated_recurrence_backward(x, gate, states, grad_out, grad_last, lens, blend, reverse, *want, workspace, _get,
                                                     _stream(index))
    if status:
        _check(status, "dc1d_gated_recurrence_backward")
    return {n: g for n, g in zip(("x", "gate", "state"), got) if g is not None}


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
