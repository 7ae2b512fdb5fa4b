"""f64 oracles of the decoder calls (include/vattn_decoder.h), with bounds of
what rounding may change -- TEST INFRASTRUCTURE ONLY, NumPy, independent of
the library.

Bounds take u, the largest relative error of one rounding to the tensors'
type (half an epsilon), and follow the sums term by term.
"""
from __future__ import annotations

import numpy as np

F32 = 2.0 ** -24  # relative error of one f32 rounding


def angles(positions, rope_dims, base=10000.0, factors=None):
    """theta[..., i] = position * base^(-2 i / rope_dims) / factors[i]."""
    i = np.arange(rope_dims // 2, dtype=np.float64)
    inv = np.power(float(base), -2.0 * i / max(rope_dims, 1))
    if factors is not None:
        inv = inv / np.asarray(factors, np.float64)[: rope_dims // 2]
    return np.asarray(positions, np.float64)[..., None] * inv


def turn(x, theta, inverse=False):
    """The NeoX rotation of x [..., D] by theta [..., half]."""
    half = theta.shape[-1]
    c, s = np.cos(theta), np.sin(theta) * (-1.0 if inverse else 1.0)
    a, b = x[..., :half], x[..., half:2 * half]
    return np.concatenate([a * c - b * s, a * s + b * c, x[..., 2 * half:]], -1)


def qk_norm_rope(x, weight, positions, rope_dims, base=10000.0, factors=None, eps=1e-6):
    """x [B, H, N, D], positions [B, N] -> (out, bound of |f32 result - out|
    before the last rounding)."""
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[-1]) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r * w
    theta = angles(positions, rope_dims, base, factors)[:, None]
    half = theta.shape[-1]
    # the row's sum of D squares carries at most D + 2 roundings, r half of
    # that, the product and the turn a few more; the angle a few 2^-24
    size = np.abs(y)
    pair = size[..., :half] + size[..., half:2 * half]
    size = np.concatenate([pair, pair, size[..., 2 * half:]], -1)
    return turn(y, theta), (x.shape[-1] / 2 + 16) * F32 * size


def qk_norm_rope_backward(g, x, weight, positions, rope_dims, base=10000.0, factors=None, eps=1e-6):
    """(dx, dw, bound of dx before its rounding, bound of dw)."""
    g, x = np.asarray(g, np.float64), np.asarray(x, np.float64)
    D = x.shape[-1]
    w = np.ones(D) if weight is None else np.asarray(weight, np.float64)
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    theta = angles(positions, rope_dims, base, factors)[:, None]
    half = theta.shape[-1]
    gy = turn(g, theta, inverse=True)
    gw = gy * w
    dx = r * gw - x * r ** 3 / D * (gw * x).sum(-1, keepdims=True)
    dw = (gy * x * r).sum((0, 1, 2))
    size = np.abs(g)
    pair = size[..., :half] + size[..., half:2 * half]
    size = np.concatenate([pair, pair, size[..., 2 * half:]], -1)  # of gy before any cancellation
    sw = size * np.abs(w)
    few = (1.5 * D + 32) * F32
    dx_bound = few * (r * sw + np.abs(x) * r ** 3 / D * (sw * np.abs(x)).sum(-1, keepdims=True))
    rows = int(np.prod(x.shape[:3]))
    dw_bound = (D / 2 + 32 + rows) * F32 * (size * np.abs(x) * r).sum((0, 1, 2))
    return dx, dw, dx_bound, dw_bound


def window_visible(n_queries, n_keys, window, n_sinks, kv_len, q_start):
    """[n_queries, n_keys] of one sequence."""
    length = n_keys if kv_len is None else min(max(int(kv_len), 0), n_keys)
    start = length - n_queries if q_start is None else int(q_start)
    p = (start + np.arange(n_queries))[:, None]
    j = np.arange(n_keys)[None, :]
    seen = (j <= p) & (p < length)
    if window is not None:
        seen &= (j > p - window) | (j < n_sinks)
    return seen


def cached_visible(n_tokens, n_keys, window, n_sinks, kv_len, words):
    """[n_tokens, n_keys] of one sequence; words: ancestor bits or None."""
    length = min(max(int(kv_len), 0), n_keys)
    base = length - n_tokens
    words = [(2 << t) - 1 for t in range(n_tokens)] if words is None else \
        [int(x) & ((1 << n_tokens) - 1) for x in words]
    seen = np.zeros((n_tokens, n_keys), bool)
    for t, word in enumerate(words):
        if word == 0 or base + t < 0:
            continue
        p = base + bin(word).count("1") - 1
        for j in range(length):
            at = j
            if j >= base:
                if not (word >> (j - base)) & 1:
                    continue
                at = base + bin(words[j - base]).count("1") - 1
            seen[t, j] = window is None or at > p - window or at < n_sinks
    return seen


def attention(q, k, v, seen, scale, u):
    """q [B, H, M, D], k, v [B, K, N, D], seen [B, M, N].  (out, lse, weights
    [B, H, M, N], bound of out, relative bound of the weights, bound of lse)
    with what is not seen left out of every sum."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    B, H, M, D = q.shape
    group = H // k.shape[1]
    out, lse = np.zeros_like(q), np.full((B, H, M), -np.inf)
    weights = np.zeros((B, H, M, k.shape[2]))
    bound, score, lse_bound = np.zeros_like(q), np.zeros((B, H, M, 1)), np.zeros((B, H, M))
    for b in range(B):
        kept = seen[b].any(0)
        for h in range(H):
            kk = np.where(kept[:, None], k[b, h // group], 0.0)
            vv = np.where(kept[:, None], v[b, h // group], 0.0)
            live = seen[b].any(1)
            qq = np.where(live[:, None], q[b, h], 0.0)
            x = np.where(seen[b], qq @ kk.T * scale, -np.inf)
            m = np.where(live, x.max(1, initial=-np.inf), 0.0)[:, None]
            e = np.exp(x - m)
            l = e.sum(1, keepdims=True)
            w = e / np.where(l > 0, l, 1.0)
            weights[b, h] = w
            out[b, h] = w @ vv
            lse[b, h] = np.where(live, m[:, 0] + np.log(np.where(l > 0, l, 1.0))[:, 0], -np.inf)
            # a score is a sum of D products, each rounded (or cut, twice as
            # much) to f32 on the way, then a scale and an exponential
            s = (2 * D + 8) * F32 * np.where(seen[b], np.abs(qq) @ np.abs(kk).T * scale, 0).max(1, initial=0)[:, None]
            s = 2 * s + 2.0 ** -20
            score[b, h] = s
            size = w @ np.abs(vv)
            # each weight is rounded to the type, the sums (of the weights
            # and of the products) carry an f32 rounding or two per term, and
            # the result is rounded once
            many = (4 * seen[b].sum(1)[:, None] + 64) * F32
            bound[b, h] = u * np.abs(out[b, h]) + (u + s + many) * size * (1 + u)
            lse_bound[b, h] = np.where(live, s[:, 0] + many[:, 0] + 4 * F32 * np.abs(np.where(live, lse[b, h], 0)), 0)
    return out, lse, weights, bound, score, lse_bound


def attention_backward(dout, q, k, v, out, weights, seen, scale, u, out_bound, score):
    """((dq, dk, dv), (their bounds)) from the forward call's values."""
    dout, q, k, v = (np.asarray(a, np.float64) for a in (dout, q, k, v))
    B, H, M, D = q.shape
    group = H // k.shape[1]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    bq, bk, bv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        kept, live = seen[b].any(0)[:, None], seen[b].any(1)[:, None]
        for h in range(H):
            g = h // group
            kk, vv = np.where(kept, k[b, g], 0.0), np.where(kept, v[b, g], 0.0)
            qq, do = np.where(live, q[b, h], 0.0), np.where(live, dout[b, h], 0.0)
            w, s = weights[b, h], score[b, h]
            dp, delta = do @ vv.T, (do * out[b, h]).sum(1, keepdims=True)
            ds = w * (dp - delta)
            dq[b, h] = ds @ kk * scale
            dk[b, g] += ds.T @ qq * scale
            dv[b, g] += w.T @ do
            # error of ds: its rounding, the weight's, the two sums of D
            # products, and delta from the rounded out
            sums = (2 * D + 8) * F32 * (np.abs(do) @ np.abs(vv).T + (np.abs(do) * np.abs(out[b, h])).sum(1, keepdims=True))
            e = w * ((u + s + 8 * F32) * np.abs(dp - delta) + (1 + s + u) * (sums + (np.abs(do) * out_bound[b, h]).sum(1, keepdims=True)))
            many = (2 * (seen[b].sum() and max(seen[b].sum(0).max() * group, seen[b].sum(1).max())) + 64) * F32
            bq[b, h] = e @ np.abs(kk) * scale + many * (np.abs(ds) @ np.abs(kk)) * scale
            bk[b, g] += e.T @ np.abs(qq) * scale + many * (np.abs(ds).T @ np.abs(qq)) * scale
            bv[b, g] += (w * (u + s + many)).T @ np.abs(do)
    return (dq, dk, dv), tuple(x * (1 + u) + u * np.abs(y) for x, y in ((bq, dq), (bk, dk), (bv, dv)))
