"""Decoder-layer calls on torch tensors: q/k norm with rotation, causal
attention under a sliding window with its gradients, attention of new tokens
over a cache (C ABI: include/vattn_decoder.h).

Tensors are ``[batch, heads, rows, head_dim]`` with a contiguous last
dimension and any strides otherwise, so views of a packed projection
``[batch, rows, heads, head_dim]`` (``.transpose(1, 2)``) and of a cache go in
as they are (rows that are a broadcast of one: ``forward_cached`` and
``qk_norm_rope`` only).  Every call runs on ``stream`` (default: the current torch
stream of the tensors' device) and returns without synchronising; results
that it allocates belong to that stream.  With a ``stream`` of one's own, the
inputs must be ready on it.  There is no CPU fallback.

The calls are not recorded by autograd: results carry no gradient function, also
where an input requires a gradient.  A training step calls
``backward_window`` and ``qk_norm_rope_backward`` itself, or
puts the pairs into a ``torch.autograd.Function`` of its own.
"""
from __future__ import annotations

import struct

from ._lib import _check, load_library

_ROWS = struct.Struct("=4q").pack          # vattn_rows
_QK = struct.Struct("=7q4Qdf2i4x").pack    # vattn_qk_args
_WINDOW = struct.Struct("=8q3Qfi").pack    # vattn_window_args
_LIB = None
_TORCH = None
_TENSOR = None
_DTYPES = {}
_F32 = _I32 = _I64 = None
_EMPTY = _EMPTY_LIKE = _DENSE = None


def _start():
    """First call: the library and what of torch the checks below compare with."""
    global _LIB, _TORCH, _TENSOR, _F32, _I32, _I64, _EMPTY, _EMPTY_LIKE, _DENSE
    import torch
    lib = load_library()
    _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    _TENSOR, _F32, _I32, _I64 = torch.Tensor, torch.float32, torch.int32, torch.int64
    _EMPTY, _EMPTY_LIKE, _DENSE = torch.empty, torch.empty_like, torch.contiguous_format
    _TORCH, _LIB = torch, lib


# The checks are written out in the calls: a call's whole host time is a few
# microseconds, of which a helper for each tensor would be a third.

def _first(name, t, dtypes):
    """(dtype code, dtype, device index) of a call's first tensor [batch, heads, rows, head_dim]."""
    if not isinstance(t, _TENSOR):
        raise TypeError(f"{name} must be a torch.Tensor")
    dtype = t.dtype
    code = _DTYPES.get(dtype, -1)
    if code not in dtypes:
        raise TypeError(f"{name} has unsupported dtype {dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, heads, rows, head_dim]")
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code, dtype, index


def _odd(name, t, dtype, index, shape=None):
    """Raises for a tensor that is not of the call's dtype, rank, device, or of the shape."""
    if not isinstance(t, _TENSOR):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, is {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")
    raise ValueError(f"{name} must be {'[batch, heads, rows, head_dim]' if shape is None else tuple(shape)}, "
                     f"is {tuple(t.shape)}")


def _like(name, t, dtype, index, shape):
    if not isinstance(t, _TENSOR) or t.dtype is not dtype or t.get_device() != index or t.shape != shape:
        _odd(name, t, dtype, index, shape)


def _rows(name, t):
    """vattn_rows of a tensor."""
    b, h, i, d = t.stride()
    if d != 1 and t.shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _ROWS(t.data_ptr(), b, h, i)


def _ints(name, t, dtype, shape, index):
    """Address of a contiguous integer tensor, 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, _TENSOR) or t.dtype is not dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on cuda:{index}")
    return t.data_ptr()


def _weight(name, w, dtype, dim, index):
    if not isinstance(w, _TENSOR) or (w.dtype is not _F32 and w.dtype is not dtype):
        raise TypeError(f"{name} must be a float32 or {dtype} tensor")
    if w.shape != (dim,) or w.get_device() != index or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous ({dim},) tensor on cuda:{index}")
    return w.data_ptr()


def _elsewhere(index, stream, inputs):
    """(stream handle, context) of a call that is not on the current device or
    has a stream of the caller's own.  The context makes the device current; a
    stream of the caller's own becomes the one that allocates results, so that
    their memory is not handed out while that stream still uses it, and the
    inputs are recorded on it."""
    torch = _TORCH
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index), torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _is_here(index, stream):
    """On the current device and its current stream: no context is needed."""
    return stream is None and index == _TORCH._C._cuda_getDevice()


def _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps):
    """(packed vattn_qk_args, dtype, device index, shapes of q and k)."""
    if _LIB is None:
        _start()
    code, dtype, index = _first("q", q, (0, 1, 2))
    if not isinstance(k, _TENSOR) or k.dtype is not dtype or k.get_device() != index or k.dim() != 4:
        _odd("k", k, dtype, index)
    q_shape, k_shape = q.shape, k.shape
    B, H, N, D = q_shape
    Bk, K, Nk, Dk = k_shape
    if Bk != B or Nk != N or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q_shape)}, k {tuple(k_shape)}")
    if rope_dims is None:
        rope_dims = D
    wq = wk = fptr = wcode = 0
    if q_weight is not None:
        wq = _weight("q_weight", q_weight, dtype, D, index)
        wcode = _DTYPES[q_weight.dtype]
    if k_weight is not None:
        wk = _weight("k_weight", k_weight, dtype, D, index)
        wcode = _DTYPES[k_weight.dtype]
        if q_weight is not None and q_weight.dtype is not k_weight.dtype:
            raise TypeError("q_weight and k_weight must have one dtype")
    if factors is not None:
        if not isinstance(factors, _TENSOR) or factors.dtype is not _F32:
            raise TypeError("factors must be a float32 tensor")
        if factors.get_device() != index or factors.numel() < rope_dims // 2 or not factors.is_contiguous():
            raise ValueError("factors must hold rope_dims // 2 contiguous floats on the tensors' device")
        fptr = factors.data_ptr()
    pptr = 0 if positions is None else _ints("positions", positions, _I32, (B, N), index)
    return (_QK(B, H, K, N, D, rope_dims, pos0, pptr, fptr, wq, wk, base, eps, code, wcode), dtype, index, q_shape,
            k_shape)


def _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, tree):
    """(packed vattn_window_args, dtype, device index, shapes of q and k)."""
    if _LIB is None:
        _start()
    code, dtype, index = _first("q", q, (1, 2))
    if not isinstance(k, _TENSOR) or k.dtype is not dtype or k.get_device() != index or k.dim() != 4:
        _odd("k", k, dtype, index)
    q_shape, k_shape = q.shape, k.shape
    _like("v", v, dtype, index, k_shape)
    B, H, M, D = q_shape
    Bk, K, N, Dk = k_shape
    if Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q_shape)}, k {tuple(k_shape)}")
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window must be at least 1 (None: no limit)")
    lens = 0 if kv_len is None else _ints("kv_len", kv_len, _I32, (B,), index)
    start = 0 if q_start is None else _ints("q_start", q_start, _I32, (B,), index)
    words = 0 if tree is None else _ints("tree_mask", tree, _I64, (B, M), index)
    return _WINDOW(B, H, K, M, N, D, window, n_sinks, lens, start, words, scale, code), dtype, index, q_shape, k_shape


def qk_norm_rope(q, k, q_weight=None, k_weight=None, rope_dims=None, pos0=0, positions=None,
                 base=10000.0, factors=None, eps=1e-6, q_out=None, k_out=None, stream=None):
    """RMS norm of every row of ``q`` and ``k`` (over ``head_dim``, times the
    weight) and the NeoX rotation of its first ``rope_dims`` dims (default:
    all), in one pass; returns ``(q_out, k_out)``.

    q ``[B, Hq, N, D]``, k ``[B, Hk, N, D]`` of one dtype (f32, f16, bf16);
    weights ``[D]`` in f32 or that dtype, or None.  Row n is at position
    ``pos0 + n``, or ``positions[b, n]`` (int32).  ``factors``: f32 divisors of
    the angles.  ``q_out`` / ``k_out``: where the results go (new contiguous
    tensors by default; may be q / k themselves, or rows of a cache)."""
    args, dtype, index, q_shape, k_shape = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base,
                                                    factors, eps)
    if q_out is not None:
        _like("q_out", q_out, dtype, index, q_shape)
    if k_out is not None:
        _like("k_out", k_out, dtype, index, k_shape)
    if not _is_here(index, stream):
        handle, there = _elsewhere(index, stream,
                                   (q, k, q_weight, k_weight, positions, factors, q_out, k_out))
        with there:
            return _qk_call(args, q, k, q_out, k_out, handle)
    return _qk_call(args, q, k, q_out, k_out, _TORCH._C._cuda_getCurrentRawStream(index))


def _qk_call(args, q, k, q_out, k_out, handle):
    if q_out is None:
        q_out = _EMPTY_LIKE(q, memory_format=_DENSE)
    if k_out is None:
        k_out = _EMPTY_LIKE(k, memory_format=_DENSE)
    status = _LIB.vattn_qk_norm_rope(_rows("q", q), _rows("k", k), _rows("q_out", q_out), _rows("k_out", k_out), args,
                                     handle)
    if status:
        _check(status)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope_dims=None, pos0=0,
                          positions=None, base=10000.0, factors=None, eps=1e-6, dq=None, dk=None,
                          stream=None):
    """Gradients of ``qk_norm_rope``: ``(dq, dk, dq_weight, dk_weight)`` from
    those of its results and its inputs.  The weights' gradients are f32
    ``[D]`` (None for a weight that is None), summed in a fixed order.
    ``dq`` / ``dk``: where the results go (may be dq_out or q, dk_out or k)."""
    args, dtype, index, q_shape, k_shape = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base,
                                                    factors, eps)
    _like("dq_out", dq_out, dtype, index, q_shape)
    _like("dk_out", dk_out, dtype, index, k_shape)
    if dq is not None:
        _like("dq", dq, dtype, index, q_shape)
    if dk is not None:
        _like("dk", dk, dtype, index, k_shape)
    rest = (dq_out, dk_out, q, k, dq, dk, q_weight is not None, k_weight is not None, q_shape[3])
    if not _is_here(index, stream):
        handle, there = _elsewhere(index, stream,
                                   (dq_out, dk_out, q, k, q_weight, k_weight, positions, factors, dq, dk))
        with there:
            return _qk_backward_call(args, *rest, handle)
    return _qk_backward_call(args, *rest, _TORCH._C._cuda_getCurrentRawStream(index))


def _qk_backward_call(args, dq_out, dk_out, q, k, dq, dk, with_q, with_k, dim, handle):
    if dq is None:
        dq = _EMPTY_LIKE(q, memory_format=_DENSE)
    if dk is None:
        dk = _EMPTY_LIKE(k, memory_format=_DENSE)
    dwq = _EMPTY(dim, dtype=_F32, device=q.device) if with_q else None
    dwk = _EMPTY(dim, dtype=_F32, device=q.device) if with_k else None
    status = _LIB.vattn_qk_norm_rope_backward(
        _rows("dq_out", dq_out), _rows("dk_out", dk_out), _rows("q", q), _rows("k", k), _rows("dq", dq),
        _rows("dk", dk), dwq.data_ptr() if with_q else 0, dwk.data_ptr() if with_k else 0, args, handle)
    if status:
        _check(status)
    return dq, dk, dwq, dwk


def forward_window(q, k, v, window=None, n_sinks=0, scale=1.0, kv_len=None, q_start=None, out=None,
                   return_lse=False, stream=None):
    """Causal attention under a sliding window whose first keys stay visible.

    q ``[B, Hq, M, D]``, k and v ``[B, Hk, N, D]`` in f16 or bf16, Hq a
    multiple of Hk, D a multiple of 8 up to 128.  Query row i is at position
    ``p = q_start[b] + i`` and sees the keys ``j <= p`` with ``j > p - window``
    (None: all) or ``j < n_sinks``, if ``0 <= p < kv_len[b]``; otherwise
    nothing, and its result is 0.  ``kv_len`` (int32 ``[B]``, default N) and
    ``q_start`` (int32 ``[B]``, default ``kv_len - M``: the queries end the
    sequence) stay on the device.  ``scale`` multiplies the scores (1: q is
    already scaled).  Returns ``out`` (q's dtype), with ``return_lse``
    ``(out, lse)``, lse f32 ``[B, Hq, M]`` for ``backward_window``."""
    args, dtype, index, q_shape, _ = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None)
    if out is not None:
        _like("out", out, dtype, index, q_shape)
    if not _is_here(index, stream):
        handle, there = _elsewhere(index, stream, (q, k, v, kv_len, q_start, out))
        with there:
            return _window_call(args, q, k, v, out, return_lse, q_shape, handle)
    return _window_call(args, q, k, v, out, return_lse, q_shape, _TORCH._C._cuda_getCurrentRawStream(index))


def _window_call(args, q, k, v, out, return_lse, q_shape, handle):
    if out is None:
        out = _EMPTY_LIKE(q, memory_format=_DENSE)
    lse = _EMPTY(q_shape[:3], dtype=_F32, device=q.device) if return_lse else None
    status = _LIB.vattn_forward_window(_rows("q", q), _rows("k", k), _rows("v", v), _rows("out", out),
                                       lse.data_ptr() if return_lse else 0, args, handle)
    if status:
        _check(status)
    return (out, lse) if return_lse else out


def backward_window(dout, q, k, v, out, lse, window=None, n_sinks=0, scale=1.0, kv_len=None, q_start=None,
                    dq=None, dk=None, dv=None, stream=None):
    """Gradients ``(dq, dk, dv)`` of ``forward_window`` from ``dout``, its
    inputs, its ``out`` and its ``lse``.  dk and dv are summed over the query
    heads that share a key head; the same call gives the same bits."""
    args, dtype, index, q_shape, k_shape = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None)
    _like("dout", dout, dtype, index, q_shape)
    _like("out", out, dtype, index, q_shape)
    if not isinstance(lse, _TENSOR) or lse.dtype is not _F32:
        raise TypeError("lse must be a float32 tensor")
    if lse.shape != q_shape[:3] or lse.get_device() != index or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous {tuple(q_shape[:3])} tensor on cuda:{index}")
    for name, t, shape in (("dq", dq, q_shape), ("dk", dk, k_shape), ("dv", dv, k_shape)):
        if t is not None:
            _like(name, t, dtype, index, shape)
    rest = (dout, q, k, v, out, lse, dq, dk, dv)
    if not _is_here(index, stream):
        handle, there = _elsewhere(index, stream, (dout, q, k, v, out, lse, kv_len, q_start, dq, dk, dv))
        with there:
            return _window_backward_call(args, *rest, handle)
    return _window_backward_call(args, *rest, _TORCH._C._cuda_getCurrentRawStream(index))


def _window_backward_call(args, dout, q, k, v, out, lse, dq, dk, dv, handle):
    if dq is None:
        dq = _EMPTY_LIKE(q, memory_format=_DENSE)
    if dk is None:
        dk = _EMPTY_LIKE(k, memory_format=_DENSE)
    if dv is None:
        dv = _EMPTY_LIKE(v, memory_format=_DENSE)
    status = _LIB.vattn_backward_window(
        _rows("dout", dout), _rows("q", q), _rows("k", k), _rows("v", v), _rows("out", out), lse.data_ptr(),
        _rows("dq", dq), _rows("dk", dk), _rows("dv", dv), args, handle)
    if status:
        _check(status)
    return dq, dk, dv


def forward_cached(q, k_cache, v_cache, kv_len, tree_mask=None, window=None, n_sinks=0, scale=1.0, out=None,
                   stream=None):
    """Attention of the newest T <= 64 tokens of each sequence over its cache.

    q ``[B, Hq, T, D]``, caches ``[B, Hk, N, D]`` (f16 or bf16) whose first
    ``kv_len[b]`` rows (int32 ``[B]``, the T new ones last) are in use.
    ``tree_mask`` (int64 ``[B, T]``): bit u of word t says that new token u is
    an ancestor of t or t itself; a token's position is that of the first new
    token plus the number of its ancestors.  None: the new tokens follow each
    other.  Window, first keys and scale as in ``forward_window``."""
    if kv_len is None:
        raise TypeError("kv_len must be an int32 tensor")
    args, dtype, index, q_shape, _ = _window_args(q, k_cache, v_cache, window, n_sinks, scale, kv_len, None,
                                                  tree_mask)
    if out is not None:
        _like("out", out, dtype, index, q_shape)
    if not _is_here(index, stream):
        handle, there = _elsewhere(index, stream, (q, k_cache, v_cache, kv_len, tree_mask, out))
        with there:
            return _cached_call(args, q, k_cache, v_cache, out, handle)
    return _cached_call(args, q, k_cache, v_cache, out, _TORCH._C._cuda_getCurrentRawStream(index))


def _cached_call(args, q, k_cache, v_cache, out, handle):
    if out is None:
        out = _EMPTY_LIKE(q, memory_format=_DENSE)
    status = _LIB.vattn_forward_cached(_rows("q", q), _rows("k_cache", k_cache), _rows("v_cache", v_cache),
                                       _rows("out", out), args, handle)
    if status:
        _check(status)
    return out
