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

import struct

from ._lib import _check, load_library

_ROWS = struct.Struct("=4q")          # vattn_rows
_QK = struct.Struct("=7q4Qdf2i4x")    # vattn_qk_args
_WINDOW = struct.Struct("=8q3Qfi")    # vattn_window_args

_TORCH = None
_DTYPES = {}


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _DTYPES.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
        _TORCH = torch
    return _TORCH


def _tensor(name, t, dtypes, device=None):
    """Type, rank and device of a [batch, heads, rows, head_dim] tensor; its dtype code."""
    torch = _TORCH
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    code = _DTYPES.get(t.dtype, -1)
    if code not in dtypes:
        raise TypeError(f"{name} has unsupported dtype {t.dtype}")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [batch, heads, rows, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, is on {t.device}")
    return code


def _like(name, t, ref, shape, code):
    """t has ref's dtype and device, and the shape."""
    if _tensor(name, t, (code,), ref.device) != code or t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, is {tuple(t.shape)}")


def _rows(name, t):
    """vattn_rows of a tensor."""
    s = t.stride()
    if s[3] != 1 and t.shape[3] > 1 and t.numel() > 0:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return _ROWS.pack(t.data_ptr(), s[0], s[1], s[2])


def _ints(name, t, dtype, shape, device):
    """Address of a contiguous integer tensor, 0 for None."""
    if t is None:
        return 0
    if not isinstance(t, _TORCH.Tensor) or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} tensor")
    if t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} tensor on {device}")
    return t.data_ptr()


class _On:
    """The device and stream of a call: makes the tensors' device current
    where it is not, and a caller's own stream the one that allocates results
    (so that their memory is not handed out while that stream still uses it)
    and that the inputs are recorded on."""

    def __init__(self, device, stream, inputs):
        torch = _TORCH
        if stream is None:
            self.stream = torch.cuda.current_stream(device)
            self.ctx = None if device.index == torch.cuda.current_device() else torch.cuda.device(device)
        else:
            if stream.device != device:
                raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
            self.stream = stream
            self.ctx = torch.cuda.stream(stream)  # makes the stream's device current too
            for t in inputs:
                if t is not None:
                    t.record_stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.stream.cuda_stream

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code):
    torch = _TORCH
    B, H, N, D = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}")
    if rope_dims is None:
        rope_dims = D
    wcode = 0
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is None:
            continue
        if not isinstance(w, torch.Tensor) or w.dtype not in (torch.float32, q.dtype):
            raise TypeError(f"{name} must be a float32 or {q.dtype} tensor")
        if w.shape != (D,) or w.device != q.device or not w.is_contiguous():
            raise ValueError(f"{name} must be a contiguous ({D},) tensor on {q.device}")
        wcode = _DTYPES[w.dtype]
    if q_weight is not None and k_weight is not None and q_weight.dtype != k_weight.dtype:
        raise TypeError("q_weight and k_weight must have one dtype")
    fptr = 0
    if factors is not None:
        if not isinstance(factors, torch.Tensor) or factors.dtype != torch.float32:
            raise TypeError("factors must be a float32 tensor")
        if factors.device != q.device or factors.numel() < rope_dims // 2 or not factors.is_contiguous():
            raise ValueError("factors must hold rope_dims // 2 contiguous floats on the tensors' device")
        fptr = factors.data_ptr()
    pptr = _ints("positions", positions, torch.int32, (B, N), q.device)
    return _QK.pack(B, H, k.shape[1], N, D, rope_dims, pos0, pptr, fptr,
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
    code = _tensor("q", q, (0, 1, 2))
    _tensor("k", k, (code,), q.device)
    args = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code)
    if q_out is not None:
        _like("q_out", q_out, q, q.shape, code)
    if k_out is not None:
        _like("k_out", k_out, q, k.shape, code)
    with _On(q.device, stream, (q, k, q_weight, k_weight, positions, factors, q_out, k_out)) as s:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if k_out is None:
            k_out = torch.empty(k.shape, dtype=q.dtype, device=q.device)
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
    code = _tensor("q", q, (0, 1, 2))
    _tensor("k", k, (code,), q.device)
    args = _qk_args(q, k, q_weight, k_weight, rope_dims, pos0, positions, base, factors, eps, code)
    _like("dq_out", dq_out, q, q.shape, code)
    _like("dk_out", dk_out, q, k.shape, code)
    if dq is not None:
        _like("dq", dq, q, q.shape, code)
    if dk is not None:
        _like("dk", dk, q, k.shape, code)
    with _On(q.device, stream,
             (dq_out, dk_out, q, k, q_weight, k_weight, positions, factors, dq, dk)) as s:
        if dq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if dk is None:
            dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
        dwq = None if q_weight is None else torch.empty(q.shape[3], dtype=torch.float32, device=q.device)
        dwk = None if k_weight is None else torch.empty(q.shape[3], dtype=torch.float32, device=q.device)
        _check(load_library().vattn_qk_norm_rope_backward(
            _rows("dq_out", dq_out), _rows("dk_out", dk_out), _rows("q", q), _rows("k", k), _rows("dq", dq),
            _rows("dk", dk), 0 if dwq is None else dwq.data_ptr(), 0 if dwk is None else dwk.data_ptr(),
            args, s))
    return dq, dk, dwq, dwk


def _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, tree, code):
    torch = _TORCH
    _tensor("k", k, (code,), q.device)
    _tensor("v", v, (code,), q.device)
    B, H, M, D = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[3] != D:
        raise ValueError(f"shape mismatch: q {tuple(q.shape)}, k {tuple(k.shape)}, v {tuple(v.shape)}")
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window must be at least 1 (None: no limit)")
    dev = q.device
    return _WINDOW.pack(B, H, k.shape[1], M, k.shape[2], D, window, n_sinks,
                        _ints("kv_len", kv_len, torch.int32, (B,), dev),
                        _ints("q_start", q_start, torch.int32, (B,), dev),
                        _ints("tree_mask", tree, torch.int64, (B, M), dev), scale, code)


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
    code = _tensor("q", q, (1, 2))
    args = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None, code)
    if out is not None:
        _like("out", out, q, q.shape, code)
    with _On(q.device, stream, (q, k, v, kv_len, q_start, out)) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=q.device) if return_lse else None
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
    code = _tensor("q", q, (1, 2))
    args = _window_args(q, k, v, window, n_sinks, scale, kv_len, q_start, None, code)
    _like("dout", dout, q, q.shape, code)
    _like("out", out, q, q.shape, code)
    if not isinstance(lse, torch.Tensor) or lse.dtype != torch.float32:
        raise TypeError("lse must be a float32 tensor")
    if lse.shape != q.shape[:3] or lse.device != q.device or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous {tuple(q.shape[:3])} tensor on {q.device}")
    for name, t, ref in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _like(name, t, q, ref.shape, code)
    with _On(q.device, stream, (dout, q, k, v, out, lse, kv_len, q_start, dq, dk, dv)) as s:
        if dq is None:
            dq = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if dk is None:
            dk = torch.empty(k.shape, dtype=q.dtype, device=q.device)
        if dv is None:
            dv = torch.empty(v.shape, dtype=q.dtype, device=q.device)
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
    torch = _torch()
    code = _tensor("q", q, (1, 2))
    if kv_len is None:
        raise TypeError("kv_len must be an int32 tensor")
    args = _window_args(q, k_cache, v_cache, window, n_sinks, scale, kv_len, None, tree_mask, code)
    if out is not None:
        _like("out", out, q, q.shape, code)
    with _On(q.device, stream, (q, k_cache, v_cache, kv_len, tree_mask, out)) as s:
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _check(load_library().vattn_forward_cached(_rows("q", q), _rows("k_cache", k_cache),
                                                   _rows("v_cache", v_cache), _rows("out", out), args, s))
    return out
