"""Decoder-layer calls on torch tensors: q/k norm with rotation, causal
attention under a sliding window with its gradients, attention of new tokens
over a cache (C ABI: include/vattn_decoder.h).

Tensors are ``[batch, heads, rows, head_dim]`` with a contiguous last
dimension and any strides otherwise, so views of a packed projection
``[batch, rows, heads, head_dim]`` (``.transpose(1, 2)``) and of a cache go in
as they are.  Every call runs on ``stream`` (default: the current torch
stream of the tensors' device) and returns without synchronising; results
that it allocates belong to that stream.  With a ``stream`` of one's own, the
inputs must be ready on it.  There is no CPU fallback.
"""
from __future__ import annotations

import contextlib
import struct

from ._lib import _check, load_library

_ROWS = struct.Struct("=4q").pack          # vattn_rows
_QK = struct.Struct("=7q4Qdf2i4x").pack    # vattn_qk_args
_WINDOW = struct.Struct("=8q3Qfi").pack    # vattn_window_args
_HERE = contextlib.nullcontext()

_TORCH = None
_DTYPES = {}


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        _TORCH = torch
    return _TORCH


def _tensor(name, t, dtypes):
    """Type and rank of a [batch, heads, rows, head_dim] CUDA tensor: (dtype code, device index)."""
    if not isinstance(t, _TORCH.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype, -1)
    if code not in dtypes:
        raise TypeError(f"{name} has unsupported dtype {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, heads, rows, head_dim]")
    index = t.get_device()
    if index < 0 or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return code, index


def _like(name, t, ref, shape=None):
    """t has ref's dtype and device, and the shape (default: ref's)."""
    if not isinstance(t, _TORCH.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != ref.dtype:
        raise TypeError(f"{name} must be {ref.dtype}, is {t.dtype}")
    if t.get_device() != ref.get_device():
        raise ValueError(f"{name} must be on {ref.device}, is on {t.device}")
    if t.shape != (ref.shape if shape is None else shape):
        raise ValueError(f"{name} must be {tuple(ref.shape if shape is None else shape)}, is {tuple(t.shape)}")


def _rows(name, t):
    """vattn_rows of a tensor."""
    b, h, i, d = t.stride()
    if d != 1 and t.shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _ROWS(t.data_ptr(), b, h, i)


def _ints(name, t, dtype, shape, ref):
    """Address of a contiguous integer tensor on ref's device, 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, _TORCH.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or t.get_device() != ref.get_device() or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {ref.device}")
    return t.data_ptr()


def _on(index, stream, inputs):
    """(stream handle, context) of a call on device `index`.  The context makes
    the tensors' device current where it is not.  A stream of the caller's own
    becomes the one that allocates results, so that their memory is not handed
    out while that stream still uses it, and the inputs are recorded on it."""
    torch = _TORCH
    if stream is None:
        # the handle without a Stream object around it: microseconds of a call
        handle = torch._C._cuda_getCurrentRawStream(index)
        return handle, _HERE if index == torch._C._cuda_getDevice() else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{index}")
    for t in inputs:
        if t is not None:
            t.record_stream(stream)
    return stream.cuda_stream, torch.cuda.stream(stream)


def _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code):
    torch = _TORCH
    B, H, N, D = q.shape
    Bk, K, Nk, Dk = k.shape
    if Bk != B or Nk != N or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    if rope_dims is None:
        rope_dims = D
    wcode = 0
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, q.dtype):
            raise TypeError(f"{name} must be a float32 or {q.dtype} tensor")
        if w.shape != (D,) or w.get_device() != q.get_device() or not w.is_contiguous():
            raise ValueError(f"{name} must be a contiguous ({D},) tensor on {q.device}")
        wcode = _DTYPES[w.dtype]
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    fptr = 0
    if factors is not None:
        if not isinstance(factors, torch.Tensor) or factors.dtype != torch.float32:
            raise TypeError("factors must be a float32 tensor")
        if factors.get_device() != q.get_device() or factors.numel() < rope_dims // 2 or not factors.is_contiguous():
            raise ValueError("factors must hold rope_dims // 2 contiguous floats on the tensors' device")
        fptr = factors.data_ptr()
    pptr = _ints("positions", positions, torch.int32, (B, N), q)
    return _QK(B, H, K, N, D, rope_dims, pos0, pptr, fptr,
               0 if q_weight is None else q_weight.data_ptr(),
               0 if k_weight is None else k_weight.data_ptr(), base, eps, code, wcode)


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
    torch = _torch()
    code, index = _tensor("q", q, (0, 1, 2))
    if _tensor("k", k, (code,))[1] != index:
        raise ValueError("q and k must be on one device")
    args = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code)
    if q_out is not None:
        _like("q_out", q_out, q)
    if k_out is not None:
        _like("k_out", k_out, k)
    s, ctx = _on(index, stream, (q, k, q_weight, k_weight, positions, factors, q_out, k_out))
    with ctx:
        if q_out is None:
            q_out = q.new_empty(q.shape)
        if k_out is None:
            k_out = k.new_empty(k.shape)
        _check(load_library().vattn_qk_norm_rope(_rows("q", q), _rows("k", k), _rows("q_out", q_out),
                                                 _rows("k_out", k_out), args, s))
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight=None, k_weight=None, rope_dims=None, pos0=0,
                          positions=None, base=10000.0, factors=None, eps=1e-6, dq=None, dk=None,
                          stream=None):
    """Gradients of ``qk_norm_rope``: ``(dq, dk, dq_weight, dk_weight)`` from
    those of its results and its inputs.  The weights' gradients are f32
    ``[D]`` (None for a weight that is None), summed in a fixed order.
    ``dq`` / ``dk``: where the results go (may be dq_out or q, dk_out or k)."""
    torch = _torch()
    code, index = _tensor("q", q, (0, 1, 2))
    if _tensor("k", k, (code,))[1] != index:
        raise ValueError("q and k must be on one device")
    args = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code)
    _like("dq_out", dq_out, q)
    _like("dk_out", dk_out, k)
    if dq is not None:
        _like("dq", dq, q)
    if dk is not None:
        _like("dk", dk, k)
    s, ctx = _on(index, stream, (dq_out, dk_out, q, k, q_weight, k_weight, positions, factors, dq, dk))
    with ctx:
        if dq is None:
            dq = q.new_empty(q.shape)
        if dk is None:
            dk = k.new_empty(k.shape)
        dwq = None if q_weight is None else q.new_empty(q.shape[3], dtype=torch.float32)
        dwk = None if k_weight is None else q.new_empty(q.shape[3], dtype=torch.float32)
        _check(load_library().vattn_qk_norm_rope_backward(
            _rows("dq_out", dq_out), _rows("dk_out", dk_out), _rows("q", q), _rows("k", k), _rows("dq", dq),
            _rows("dk", dk), 0 if dwq is None else dwq.data_ptr(), 0 if dwk is None else dwk.data_ptr(),
            args, s))
    return dq, dk, dwq, dwk


def _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, tree):
    """(device index, packed vattn_window_args)."""
    torch = _TORCH
    code, index = _tensor("q", q, (1, 2))
    if _tensor("k", k, (code,))[1] != index or _tensor("v", v, (code,))[1] != index:
        raise ValueError("q, k and v must be on one device")
    B, H, M, D = q.shape
    Bk, K, N, Dk = k.shape
    if k.shape != v.shape or Bk != B or Dk != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window must be at least 1 (None: no limit)")
    return index, _WINDOW(B, H, K, M, N, D, window, n_sinks, _ints("kv_len", kv_len, torch.int32, (B,), q),
                          _ints("q_start", q_start, torch.int32, (B,), q),
                          _ints("tree_mask", tree, torch.int64, (B, M), q), scale, code)


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
    torch = _torch()
    index, args = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None)
    if out is not None:
        _like("out", out, q)
    s, ctx = _on(index, stream, (q, k, v, kv_len, q_start, out))
    with ctx:
        if out is None:
            out = q.new_empty(q.shape)
        lse = q.new_empty(q.shape[:3], dtype=torch.float32) if return_lse else None
        _check(load_library().vattn_forward_window(_rows("q", q), _rows("k", k), _rows("v", v),
                                                   _rows("out", out), lse.data_ptr() if return_lse else 0,
                                                   args, s))
    return (out, lse) if return_lse else out


def backward_window(dout, q, k, v, out, lse, window=None, n_sinks=0, scale=1.0, kv_len=None, q_start=None,
                    dq=None, dk=None, dv=None, stream=None):
    """Gradients ``(dq, dk, dv)`` of ``forward_window`` from ``dout``, its
    inputs, its ``out`` and its ``lse``.  dk and dv are summed over the query
    heads that share a key head; the same call gives the same bits."""
    torch = _torch()
    index, args = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None)
    _like("dout", dout, q)
    _like("out", out, q)
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32:
        raise TypeError("lse must be a float32 tensor")
    if lse.shape != q.shape[:3] or lse.get_device() != index or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous {tuple(q.shape[:3])} tensor on {q.device}")
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _like(name, t, ref)
    s, ctx = _on(index, stream, (dout, q, k, v, out, lse, kv_len, q_start, dq, dk, dv))
    with ctx:
        if dq is None:
            dq = q.new_empty(q.shape)
        if dk is None:
            dk = k.new_empty(k.shape)
        if dv is None:
            dv = v.new_empty(v.shape)
        _check(load_library().vattn_backward_window(
            _rows("dout", dout), _rows("q", q), _rows("k", k), _rows("v", v), _rows("out", out),
            lse.data_ptr(), _rows("dq", dq), _rows("dk", dk), _rows("dv", dv), args, s))
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
    _torch()
    if kv_len is None:
        raise TypeError("kv_len must be an int32 tensor")
    index, args = _window_args(q, k_cache, v_cache, window, n_sinks, scale, kv_len, None, tree_mask)
    if out is not None:
        _like("out", out, q)
    s, ctx = _on(index, stream, (q, k_cache, v_cache, kv_len, tree_mask, out))
    with ctx:
        if out is None:
            out = q.new_empty(q.shape)
        _check(load_library().vattn_forward_cached(_rows("q", q), _rows("k_cache", k_cache),
                                                   _rows("v_cache", v_cache), _rows("out", out), args, s))
    return out
