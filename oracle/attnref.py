"""Plain CPU reference for rotary positions, the paged cache and the attention over it (test
infrastructure): fp64, one head and one row at a time, no blocking.  It shares no code with the
GPU library.

  rope       -- pair i of a head's first R dims times mscale * exp(+-i pos freq[i])
  e4m3_*     -- the 256 values of the 8-bit format and rounding to nearest, ties to even
  append     -- tokens to their slots of [pages][heads][page size][dim] arrays
  attention  -- softmax over the keys that a row sees, and the scales of its error bound
"""

from __future__ import annotations

import numpy as np


def rope(x, pos, freq, *, interleaved=False, mscale=1.0, inverse=False):
    """fp64 [T][H][D]: x with the first 2 * len(freq) dims of every head rotated."""
    y = np.asarray(x, dtype=np.float64).copy()
    half = len(freq)
    ang = np.asarray(pos, dtype=np.float64)[:, None] * np.asarray(freq, dtype=np.float64)[None, :]
    c, s = np.cos(ang) * mscale, np.sin(ang) * mscale * (-1.0 if inverse else 1.0)
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b = y[:, :, ia].copy(), y[:, :, ib].copy()
        y[:, :, ia] = a * c[:, i, None] - b * s[:, i, None]
        y[:, :, ib] = b * c[:, i, None] + a * s[:, i, None]
    return y


def e4m3_values():
    """The value of each of the 256 codes (0x7f and 0xff: NaN)."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        e, m = (code >> 3) & 0xF, code & 7
        if e == 15 and m == 7:
            out[code] = np.nan
        elif e == 0:
            out[code] = sign * m * 2.0 ** -9
        else:
            out[code] = sign * (1 + m / 8) * 2.0 ** (e - 7)
    return out


def e4m3_round(x):
    """uint8 codes: nearest, ties to the even code, saturated at +-448; NaN gives a NaN code."""
    x = np.asarray(x, dtype=np.float64)
    vals = e4m3_values()[:127]  # 0 .. 448, increasing
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(vals, np.nan_to_num(a)), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d = (vals[hi] - a) - (a - vals[lo])  # > 0: the lower is nearer
    code = np.where(d > 0, lo, np.where(d < 0, hi, np.where(hi % 2 == 0, hi, lo))).astype(np.uint8)
    code = np.where(np.isnan(x), 0x7F, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def append(cache, rows, slots):
    """cache [pages][heads][page size][dim] with rows[t] ([heads][dim]) at slot[t]; others skipped."""
    out = cache.copy()
    pages, _, ps, _ = cache.shape
    for t, s in enumerate(np.asarray(slots)):
        if 0 <= s < pages * ps:
            out[s // ps, :, s % ps] = rows[t]
    return out


def attention(q, k_cache, v_cache, table, kv_len, q_start, *, scale, window=0, k_scale=None, v_scale=None):
    """(out fp64 [T][Hq][D], size [T][Hq][D], wobble [T][Hq]): out; the weighted mean of |v|, the scale of
    relative errors of the weights; and the largest sum of |scale q_d k_d| over the keys seen, the scale
    of the scores' rounding errors.  Rows of no sequence are NaN; values beyond what a row sees are never touched."""
    q = np.asarray(q, dtype=np.float64)
    t_all, hq, d = q.shape
    hkv, ps = k_cache.shape[1], k_cache.shape[2]
    out, size, wobble = np.full((t_all, hq, d), np.nan), np.zeros((t_all, hq, d)), np.zeros((t_all, hq))
    for b in range(len(kv_len)):
        n = int(q_start[b + 1]) - int(q_start[b])
        length = int(kv_len[b])
        if n == 0:
            continue
        ids = [int(p) for p in table[b, :-(-length // ps)]]
        keys = {}
        for g in range(hkv):
            k = np.concatenate([k_cache[p, g] for p in ids] or [np.zeros((0, d))])[:length].astype(np.float64)
            v = np.concatenate([v_cache[p, g] for p in ids] or [np.zeros((0, d))])[:length].astype(np.float64)
            keys[g] = (k * (1.0 if k_scale is None else float(k_scale[g])),
                       v * (1.0 if v_scale is None else float(v_scale[g])))
        for i in range(n):
            p, t = length - n + i, int(q_start[b]) + i
            lo = max(0, p + 1 - window) if window else 0
            for h in range(hq):
                if p < lo or p < 0:
                    out[t, h] = 0.0
                    continue
                k, v = (x[lo:p + 1] for x in keys[h // (hq // hkv)])
                s = k @ q[t, h] * scale
                e = np.exp(s - s.max())
                w = e / e.sum()
                out[t, h] = w @ v
                size[t, h] = w @ np.abs(v)
                wobble[t, h] = (np.abs(k) @ np.abs(q[t, h])).max() * scale
    return out, size, wobble
