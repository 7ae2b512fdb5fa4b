"""f64 oracles of the serving calls (include/vattn_serving.h), with bounds of
what rounding may change -- TEST INFRASTRUCTURE ONLY, NumPy, independent of
the library.
"""
from __future__ import annotations

import numpy as np

from . import decoder as od

F32 = od.F32
F16 = 2.0 ** -11  # relative error of one f16 rounding
TOP, MIN_EXPONENT = 448.0, -32


def e4m3_round(x):
    """To nearest even among the values of e4m3: steps of 2^(e - 3) at 2^e .. 2^(e + 1),
    2^-9 below 2^-6, 448 the largest (beyond it: 448); NaN stays, infinities become NaN."""
    x = np.asarray(x, np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    e = np.floor(np.log2(np.maximum(a, 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    y = np.minimum(np.rint(a / step) * step, TOP)
    return np.where(np.isfinite(x), np.copysign(y, x), np.nan)


def scale_for(most):
    """The smallest power of two s >= 2^-32 with most <= 448 s."""
    if most <= TOP * 2.0 ** MIN_EXPONENT:
        return 2.0 ** MIN_EXPONENT
    m, e = np.frexp(most / TOP)  # = m 2^e, 1/2 <= m < 1 (448 is 7 * 2^6: the quotient of a power of two by it is exact)
    return 2.0 ** (e if m > 0.5 else e - 1)


class Cache:
    """The values of one pool ([n_pages, H, page, D], in units of the scales) and its
    scales [n_pages, H], as appends leave them; lo and hi are the two values that a
    rounding of a value known up to an error may give."""

    def __init__(self, values, scales):
        self.lo = np.array(values, np.float64)
        self.hi = self.lo.copy()
        self.scale = np.array(scales, np.float64)
        self.loose = np.zeros(self.scale.shape, bool)  # scales that rounding may have put a power further

    def append(self, table, kv_len, x, error):
        """x [H, n, D]: the last n rows of a sequence of kv_len rows, known up to `error`."""
        page = self.lo.shape[2]
        n = x.shape[1]
        row = kv_len - n
        i = max(0, -row)
        while i < n and (row + i) // page < len(table):
            r = row + i
            take = min(page - r % page, n - i)
            P, at = int(table[r // page]), r % page
            if 0 <= P < self.lo.shape[0]:
                for h in range(x.shape[0]):
                    part, err = x[h, i:i + take], error[h, i:i + take]
                    ok = np.isfinite(part)
                    most = np.abs(part[ok]).max(initial=0.0)
                    slack = err[ok].max(initial=0.0)
                    need = scale_for(most)
                    self.loose[P, h] |= scale_for(most + slack) != scale_for(max(most - slack, 0.0))
                    old = self.scale[P, h]
                    scale = need if at == 0 else max(old, need)
                    if at and scale != old:
                        for pool in (self.lo, self.hi):
                            pool[P, h, :at] = e4m3_round(pool[P, h, :at] * (old / scale))
                    self.scale[P, h] = scale
                    self.lo[P, h, at:at + take] = e4m3_round((part - err) / scale)
                    self.hi[P, h, at:at + take] = e4m3_round((part + err) / scale)
            i += take


def rotated(x, positions, rope_dims, base=10000.0, factors=None):
    """(the NeoX rotation of x [H, n, D] at positions [n], bound of an f32 computation's error)."""
    theta = od.angles(positions, rope_dims, base, factors)
    half = theta.shape[-1]
    y = od.turn(np.asarray(x, np.float64), theta)
    size = np.abs(x)
    pair = size[..., :half] + size[..., half:2 * half]
    # angles, sines and cosines to about 2^-23 together, two products and their sum
    error = 6 * F32 * np.concatenate([pair, pair, np.zeros_like(size[..., 2 * half:])], -1)
    return y, np.where(np.isfinite(error), error, 0.0)


def gathered(pages, scales, table, n_rows):
    """[H, n_rows, D] values of a sequence's first rows, and which of them are there."""
    H, page, D = pages.shape[1:]
    out, here = np.zeros((H, n_rows, D)), np.zeros(n_rows, bool)
    for r0 in range(0, n_rows, page):
        P = int(table[r0 // page])
        if 0 <= P < pages.shape[0]:
            take = min(page, n_rows - r0)
            out[:, r0:r0 + take] = pages[P, :, :take] * scales[P][:, None, None]
            here[r0:r0 + take] = True
    return out, here


def paged_attention(q, k, v, v_scale, seen, scale, u):
    """q [B, H, M, D], k, v [B, K, N, D], v_scale [B, K, N] of each row's page, seen [B, M, N]
    -> (out, bound): the weights, times the scale, in f16, the result in the type of `u`."""
    out, _, w, bound, _, _ = od.attention(q, k, v, seen, scale, F16)
    group = q.shape[1] // k.shape[1]
    for b in range(q.shape[0]):
        for h in range(q.shape[1]):
            vs = np.where(seen[b].any(0), v_scale[b, h // group], 0.0)
            kept = np.where(seen[b].any(0)[:, None], np.abs(v[b, h // group]), 0.0)
            # f16 has digits down to 2^-32 of the largest weight times scale, and the
            # exponents carry the scale's logarithm, of up to 2^6
            few = (w[b, h] * vs).max(1, initial=0.0)[:, None] * 2.0 ** -32
            bound[b, h] += few * (seen[b].astype(float) @ (kept / np.where(vs > 0, vs, 1.0)[:, None]))
            bound[b, h] += 2.0 ** -17 * (w[b, h] @ kept)
    return out, bound * (1 + u) + u * np.abs(out)
