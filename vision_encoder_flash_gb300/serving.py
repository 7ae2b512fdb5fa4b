"""Calls of a server of many requests on torch tensors: causal attention over
packed prompts, a paged cache of keys and values in 8 bits, attention of new
tokens over it (C ABI: include/vattn_serving.h).

Tensors of rows as in decoder.py: ``[batch, heads, rows, head_dim]``, any
strides, last dimension contiguous.  Packed ones are a batch of 1 whose rows
are those of all sequences, sequence b's at ``cu_seqlens[b] ..
cu_seqlens[b + 1]`` (int32 ``[n_seqs + 1]`` on the device, ascending).

The cache of a layer is six tensors, which the caller allocates and keeps:
``k_pages`` and ``v_pages`` ``[n_pages, Hk, page_size, D]`` in float8_e4m3fn (or
uint8), in any layout whose rows are contiguous and start on 16 bytes;
``k_scale`` and ``v_scale`` f32 ``[n_pages, Hk]``, by which a page's values are
multiplied; ``page_table`` int32 ``[B, max_pages]``: row r of sequence b is
row ``r % page_size`` of page ``page_table[b, r // page_size]`` (an entry
outside ``[0, n_pages)`` is a page that is not there); ``kv_len`` int32 ``[B]``:
rows in use, the new ones counted.  Pages need no initial values.

Streams, devices, errors and autograd: as in decoder.py.
"""
from __future__ import annotations

import struct

from . import decoder as _d
from ._lib import _check

_PAGES = struct.Struct("=2Q6q4Q3q").pack       # vattn_pages
_APPEND = struct.Struct("=5q3Qdi4x").pack      # vattn_append_args
_BYTES = ()                                    # dtypes of a pool


# As in decoder.py the checks are written out: a call's host time is that of a few of them.

def _odd_pool(name, t, heads, dim, index):
    """Raises for a pool that is not one of the call's heads, width and device."""
    if not isinstance(t, _d._TENSOR) or t.dtype not in _BYTES:
        raise TypeError(f"{name} must be a float8_e4m3fn (or uint8) tensor")
    if t.dim() != 4 or t.shape[1] != heads or t.shape[3] != dim:
        raise ValueError(f"{name} must be [n_pages, {heads}, page_size, {dim}], is {tuple(t.shape)}")
    raise ValueError(f"{name} must be on cuda:{index}, is on {t.device}")


def _odd_floats(name, t, shape, index):
    if not isinstance(t, _d._TENSOR) or t.dtype is not _d._F32:
        raise TypeError(f"{name} must be a float32 tensor")
    raise ValueError(f"{name} must be a contiguous {shape} tensor on cuda:{index}")


def _pages(k_pages, v_pages, k_scale, v_scale, page_table, kv_len, batch, heads, dim, index):
    """Packed vattn_pages of a cache that is read or written by `batch` sequences."""
    global _BYTES
    tensor, f32, i32 = _d._TENSOR, _d._F32, _d._I32
    if not _BYTES:
        _BYTES = (_d._TORCH.float8_e4m3fn, _d._TORCH.uint8)
    if not isinstance(k_pages, tensor) or k_pages.dtype not in _BYTES or k_pages.dim() != 4 or \
            k_pages.get_device() != index:
        _odd_pool("k_pages", k_pages, heads, dim, index)
    shape = k_pages.shape
    n_pages, pool_heads, page, pool_dim = shape
    if pool_heads != heads or pool_dim != dim:
        _odd_pool("k_pages", k_pages, heads, dim, index)
    if not isinstance(v_pages, tensor) or v_pages.dtype not in _BYTES or v_pages.get_device() != index:
        _odd_pool("v_pages", v_pages, heads, dim, index)
    if v_pages.shape != shape:
        raise ValueError(f"shape mismatch: k_pages {tuple(shape)}, v_pages {tuple(v_pages.shape)}")
    scales = (n_pages, heads)
    if not isinstance(k_scale, tensor) or k_scale.dtype is not f32 or k_scale.shape != scales or \
            k_scale.get_device() != index or not k_scale.is_contiguous():
        _odd_floats("k_scale", k_scale, scales, index)
    if not isinstance(v_scale, tensor) or v_scale.dtype is not f32 or v_scale.shape != scales or \
            v_scale.get_device() != index or not v_scale.is_contiguous():
        _odd_floats("v_scale", v_scale, scales, index)
    if not isinstance(page_table, tensor) or page_table.dim() != 2:
        raise TypeError("page_table must be an int32 tensor [batch, max_pages]")
    rows, most = page_table.shape
    if rows != batch or page_table.dtype is not i32 or page_table.get_device() != index or \
            not page_table.is_contiguous():
        _d._ints("page_table", page_table, i32, (batch, most), index)
    if kv_len is None:
        raise TypeError("kv_len must be an int32 tensor")
    lens = _d._ints("kv_len", kv_len, i32, (batch,), index)
    kp, kh, kr, kd = k_pages.stride()
    vp, vh, vr, vd = v_pages.stride()
    if (kd != 1 or vd != 1) and dim > 1 and n_pages * heads * page > 0:
        raise ValueError("k_pages and v_pages must be contiguous in their last dimension")
    return _PAGES(k_pages.data_ptr(), v_pages.data_ptr(), kp, kh, kr, vp, vh, vr, k_scale.data_ptr(),
                  v_scale.data_ptr(), page_table.data_ptr(), lens, n_pages, page, most)


def _sequences(cu_seqlens, index):
    """(address, number of sequences) of cu_seqlens."""
    if not isinstance(cu_seqlens, _d._TENSOR) or cu_seqlens.dtype is not _d._I32:
        raise TypeError("cu_seqlens must be an int32 tensor")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or cu_seqlens.get_device() != index or \
            not cu_seqlens.is_contiguous():
        raise ValueError(f"cu_seqlens must be a contiguous [n_seqs + 1] tensor on cuda:{index}")
    return cu_seqlens.data_ptr(), cu_seqlens.shape[0] - 1


def append_paged(k, v, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, cu_seqlens=None, rope_dims=0,
                 positions=None, base=10000.0, factors=None, stream=None):
    """New keys and values of every sequence into the paged cache, in place.

    k, v ``[B, Hk, T, D]`` (f16 or bf16, D a multiple of 16 up to 128): T new
    tokens of each sequence; with ``cu_seqlens`` packed ``[1, Hk, total, D]``.
    They become the last rows in use: ``kv_len`` counts them already.  The first
    ``rope_dims`` dims of a key are rotated on the way (NeoX; 0: keys come
    rotated) by its row in the cache, or by ``positions`` (int32 ``[B, T]`` or
    ``[1, total]``); ``base`` and ``factors`` as in ``qk_norm_rope``.

    Values are rounded to e4m3 in units of their page's and head's scale, a
    power of two that grows with the page's values (rows written before are
    rescaled) and starts anew where the page's row 0 is written.  A page that is
    written belongs to one sequence of the call."""
    if _d._LIB is None:
        _d._start()
    code, dtype, index = _d._first("k", k, (1, 2))
    shape = k.shape
    _d._like("v", v, dtype, index, shape)
    batch, heads, tokens, dim = shape
    cu = 0
    if cu_seqlens is not None:
        if batch != 1:
            raise ValueError(f"packed k must be [1, heads, rows, head_dim], is {tuple(shape)}")
        cu, batch = _sequences(cu_seqlens, index)
    pos = 0 if positions is None else _d._ints("positions", positions, _d._I32, (shape[0], tokens), index)
    turns = 0
    if factors is not None:
        if not isinstance(factors, _d._TENSOR) or factors.dtype is not _d._F32:
            raise TypeError("factors must be a float32 tensor")
        if factors.get_device() != index or factors.numel() < rope_dims // 2 or not factors.is_contiguous():
            raise ValueError("factors must hold rope_dims // 2 contiguous floats on the tensors' device")
        turns = factors.data_ptr()
    cache = _pages(k_pages, v_pages, k_scale, v_scale, page_table, kv_len, batch, heads, dim, index)
    args = _APPEND(batch, heads, tokens, dim, rope_dims, cu, pos, turns, base, code)
    if not _d._is_here(index, stream):
        handle, there = _d._elsewhere(index, stream, (k, v, k_pages, v_pages, k_scale, v_scale, page_table, kv_len,
                                                      cu_seqlens, positions, factors))
        with there:
            return _append_call(k, v, cache, args, handle)
    return _append_call(k, v, cache, args, _d._TORCH._C._cuda_getCurrentRawStream(index))


def _append_call(k, v, cache, args, handle):
    status = _d._LIB.vattn_append_paged(_d._rows("k", k), _d._rows("v", v), cache, args, handle)
    if status:
        _check(status)


def forward_paged(q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len, tree_mask=None, window=None, n_sinks=0,
                  scale=1.0, out=None, stream=None):
    """Attention of the newest T <= 64 tokens of each sequence over its pages.

    q ``[B, Hq, T, D]`` (f16 or bf16, D a multiple of 16 up to 128), Hq a
    multiple of the cache's heads; the new tokens' keys and values are the last
    T rows in use (``append_paged`` before).  ``tree_mask``, window, first keys,
    scale and result as in ``forward_cached``."""
    if _d._LIB is None:
        _d._start()
    code, dtype, index = _d._first("q", q, (1, 2))
    shape = q.shape
    batch, q_heads, tokens, dim = shape
    if not isinstance(k_pages, _d._TENSOR) or k_pages.dim() != 4:
        raise TypeError("k_pages must be a tensor [n_pages, heads, page_size, head_dim]")
    heads = k_pages.shape[1]
    cache = _pages(k_pages, v_pages, k_scale, v_scale, page_table, kv_len, batch, heads, dim, index)
    if window is None:
        window = 0
    elif window < 1:
        raise ValueError("window must be at least 1 (None: no limit)")
    words = 0 if tree_mask is None else _d._ints("tree_mask", tree_mask, _d._I64, (batch, tokens), index)
    args = _d._WINDOW(batch, q_heads, heads, tokens, 0, dim, window, n_sinks, 0, 0, words, scale, code)
    if out is not None:
        _d._like("out", out, dtype, index, shape)
    if not _d._is_here(index, stream):
        handle, there = _d._elsewhere(index, stream, (q, k_pages, v_pages, k_scale, v_scale, page_table, kv_len,
                                                      tree_mask, out))
        with there:
            return _paged_call(q, cache, out, args, handle)
    return _paged_call(q, cache, out, args, _d._TORCH._C._cuda_getCurrentRawStream(index))


def _paged_call(q, cache, out, args, handle):
    if out is None:
        out = _d._EMPTY_LIKE(q, memory_format=_d._DENSE)
    status = _d._LIB.vattn_forward_paged(_d._rows("q", q), cache, _d._rows("out", out), args, handle)
    if status:
        _check(status)
    return out


def forward_packed(q, k, v, cu_seqlens, window=None, n_sinks=0, scale=1.0, out=None, return_lse=False, stream=None):
    """Causal attention over prompts of different lengths in one buffer.

    q ``[1, Hq, total, D]``, k and v ``[1, Hk, total, D]`` (f16 or bf16, D a
    multiple of 8 up to 128): row i of sequence b is row ``cu_seqlens[b] + i``
    and sees the rows j <= i of its own sequence with ``j > i - window`` (None:
    all) or ``j < n_sinks``.  Returns ``out`` as q, with ``return_lse`` ``(out,
    lse)``, lse f32 ``[1, Hq, total]``.  Rows in no sequence are left as they
    are (not set, in results that the call allocates)."""
    args, dtype, index, shape, k_shape = _d._window_args(q, k, v, window, n_sinks, scale, None, None, None)
    cu, n_seqs = _sequences(cu_seqlens, index)
    if out is not None:
        _d._like("out", out, dtype, index, shape)
    if not _d._is_here(index, stream):
        handle, there = _d._elsewhere(index, stream, (q, k, v, cu_seqlens, out))
        with there:
            return _packed_call(args, q, k, v, cu, n_seqs, out, return_lse, shape, handle)
    return _packed_call(args, q, k, v, cu, n_seqs, out, return_lse, shape,
                        _d._TORCH._C._cuda_getCurrentRawStream(index))


def _packed_call(args, q, k, v, cu, n_seqs, out, return_lse, shape, handle):
    if out is None:
        out = _d._EMPTY_LIKE(q, memory_format=_d._DENSE)
    lse = _d._EMPTY(shape[:3], dtype=_d._F32, device=q.device) if return_lse else None
    status = _d._LIB.vattn_forward_packed(_d._rows("q", q), _d._rows("k", k), _d._rows("v", v), _d._rows("out", out),
                                          lse.data_ptr() if return_lse else 0, cu, n_seqs, args, handle)
    if status:
        _check(status)
    return (out, lse) if return_lse else out
