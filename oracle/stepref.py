"""Plain CPU reference for a decode step with drafted tokens (test infrastructure): whole numbers in Python,
values in fp64, one element at a time where it can be.  It shares no code with the GPU library.

  norm       -- x w / sqrt(mean(x^2) + eps) of every head
  plan       -- pages given back and taken, row starts, positions, slots
  attention  -- softmax over an explicit list of keys for each row, and the scales of its error bound
  adjust     -- penalties, biases and masks on logits
"""

from __future__ import annotations

import math

import numpy as np


def norm(x, weight, eps):
    """fp64 [T][H][D]"""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def plan(kv_len, new_len, table, owned, free, count, page, rows, depth=None):
    """dict of what a step leaves behind; the arguments are not changed."""
    table, owned, free = [list(map(int, r)) for r in table], list(map(int, owned)), list(map(int, free))
    n_seq, width, pages = len(owned), len(table[0]), len(free)
    count = min(max(int(count), 0), pages)
    owned = [min(max(x, 0), width) for x in owned]
    starts, fits = [0], []
    for b in range(n_seq):
        old, new = int(kv_len[b]), int(new_len[b])
        start = min(starts[-1], rows)
        fits.append(old >= 0 and new >= 0 and old + new <= width * page and start + new <= rows)
        starts.append(starts[-1] + min(max(new, 0), rows))
    starts = [min(s, rows) for s in starts]
    need = [-(-(int(kv_len[b]) + int(new_len[b])) // page) if fits[b] else owned[b] for b in range(n_seq)]
    for b in range(n_seq):
        for j in range(need[b], owned[b]):
            if count < pages:
                free[count] = table[b][j]
                count += 1
            table[b][j] = -1
        owned[b] = min(owned[b], need[b])
    left, status, total = count, [], []
    pos, slot = [0] * rows, [-1] * rows
    for b in range(n_seq):
        lack = need[b] - owned[b]
        left -= lack
        granted = lack == 0 or left >= 0
        if granted:
            for j in range(owned[b], need[b]):
                count -= 1
                table[b][j] = free[count]
            owned[b] = need[b]
        status.append(-1 if not fits[b] else 0 if granted else lack)
        total.append(int(kv_len[b]) + int(new_len[b]) if status[b] == 0 else int(kv_len[b]))
        if status[b] < 0:
            continue
        for i in range(int(new_len[b])):
            t, at = starts[b] + i, int(kv_len[b]) + i
            pos[t] = at if depth is None else int(kv_len[b]) + int(depth[t])
            if status[b] == 0 and 0 <= table[b][at // page] < pages:
                slot[t] = table[b][at // page] * page + at % page
    return dict(q_start=starts, kv_total=total, pos=pos, slot=slot, status=status, table=table, owned=owned, free=free,
                count=count)


def seen_keys(bits, kv_len, n, window=0):
    """Key numbers that a row of a tree sees: bits is the set of new tokens (numbers) that it is to see."""
    base = kv_len - n
    bits = {j for j in bits if j < n}
    depth = max(len(bits) - 1, 0)
    lo = max(0, base + depth + 1 - window) if window else 0
    return list(range(lo, max(base, 0))) + sorted(base + j for j in bits if base + j >= 0)


def attention(q, k_cache, v_cache, table, kv_len, q_start, sees, *, scale, window=0, k_scale=None, v_scale=None):
    """(out, size, wobble) as attnref.attention gives them; sees[t]: the new tokens that row t is to see."""
    q = np.asarray(q, dtype=np.float64)
    t_all, hq, d = q.shape
    hkv, ps = k_cache.shape[1], k_cache.shape[2]
    out, size, wobble = np.full((t_all, hq, d), np.nan), np.zeros((t_all, hq, d)), np.zeros((t_all, hq))
    for b in range(len(kv_len)):
        first, n, length = int(q_start[b]), int(q_start[b + 1]) - int(q_start[b]), int(kv_len[b])
        for i in range(n):
            keys = np.array(seen_keys(sees[first + i], length, n, window), dtype=np.int64)
            pages = np.asarray(table)[b, keys // ps]
            for h in range(hq):
                g = h // (hq // hkv)
                if len(keys) == 0:
                    out[first + i, h] = 0.0
                    continue
                k = k_cache[pages, g, keys % ps].astype(np.float64) * (1.0 if k_scale is None else float(k_scale[g]))
                v = v_cache[pages, g, keys % ps].astype(np.float64) * (1.0 if v_scale is None else float(v_scale[g]))
                s = k @ q[first + i, h] * scale
                w = np.exp(s - s.max())
                w = w / w.sum()
                out[first + i, h] = w @ v
                size[first + i, h] = w @ np.abs(v)
                wobble[first + i, h] = (np.abs(k) @ np.abs(q[first + i, h])).max() * scale
    return out, size, wobble


def adjust(logits, requests=None, tokens=None, token_len=None, prompt_len=None, repetition=None, frequency=None,
           presence=None, bias=None, allowed=None):
    """(fp64 [M][V], [M][V] sum of the sizes of what was added up): bias[s]: a list of (token, value); allowed[m]: a
    set of tokens, or None."""
    x = np.asarray(logits, dtype=np.float64).copy()
    m_all, v_all = x.shape
    size = np.abs(x)
    for m in range(m_all):
        s = m if requests is None else int(requests[m])
        known = s >= 0 and (tokens is None or s < len(tokens)) and (bias is None or s < len(bias))
        if tokens is not None and known:
            length = min(max(int(token_len[s]), 0), tokens.shape[1])
            at = 0 if prompt_len is None else int(prompt_len[s])
            said = {}
            for i, t in enumerate(map(int, tokens[s, :length])):
                said[t] = said.get(t, 0) + (i >= at)
            for t, c in said.items():
                if not 0 <= t < v_all:
                    continue
                r = 1.0 if repetition is None else float(repetition[s])
                x[m, t] = x[m, t] / r if x[m, t] > 0 else x[m, t] * r
                size[m, t] = abs(x[m, t])
                if c:
                    f = 0.0 if frequency is None else float(frequency[s])
                    p = 0.0 if presence is None else float(presence[s])
                    x[m, t] -= f * c + p
                    size[m, t] += abs(f) * c + abs(p)
        if bias is not None and known:
            for t, b in {int(t): float(b) for t, b in bias[s]}.items():
                if 0 <= t < v_all:
                    x[m, t] += b
                    size[m, t] += abs(b)
        if allowed is not None and allowed[m] is not None:
            keep = np.zeros(v_all, dtype=bool)
            keep[[t for t in allowed[m]]] = True
            x[m, ~keep] = -math.inf
    return x, size
