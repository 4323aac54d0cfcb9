"""Attention of packed sequences in 64 bits, one query head at a time, with what a test needs to bound the error
of a computation in fewer bits."""
from __future__ import annotations

import numpy as np

__all__ = ["attention", "paged_rows", "tolerance"]


def attention(q, keys, values, q_start, kv_len, heads, kv_heads, head_dim, scale, causal):
    """Rows q [T, heads * head_dim]; keys[b], values[b]: [kv_len[b], kv_heads, head_dim] of sequence b.

    Returns (out, lse, spread, reach): out [T, heads, head_dim]; lse [T, heads], -inf where a row sees no key;
    spread = sum of weights * |value| (what a relative error of the weights scales with); reach [T, heads] = the
    largest scale * sum |q * k| of a row (what a relative error of the products scales with). Rows of no sequence
    are NaN."""
    T = q.shape[0]
    q = q.astype(np.float64).reshape(T, heads, head_dim)
    out = np.full((T, heads, head_dim), np.nan)
    spread, lse, reach = out.copy(), np.full((T, heads), np.nan), np.full((T, heads), np.nan)
    group = heads // kv_heads
    for b in range(len(kv_len)):
        r0, r1, L = int(q_start[b]), int(q_start[b + 1]), int(kv_len[b])
        n = r1 - r0
        for i in range(n):
            p = L - n + i
            sees = max(0, min(L, p + 1)) if causal else L
            for h in range(heads):
                t = r0 + i
                if sees == 0:
                    out[t, h], spread[t, h], lse[t, h], reach[t, h] = 0, 0, -np.inf, 0
                    continue
                k = keys[b][:sees, h // group].astype(np.float64)
                v = values[b][:sees, h // group].astype(np.float64)
                s = scale * (k @ q[t, h])
                m = s.max()
                w = np.exp(s - m)
                total = w.sum()
                w = w / total
                out[t, h] = w @ v
                spread[t, h] = w @ np.abs(v)
                lse[t, h] = m + np.log(total)
                reach[t, h] = scale * (np.abs(k) @ np.abs(q[t, h])).max()
    return out, lse, spread, reach


def paged_rows(cache, table, kv_len):
    """The keys (or values) of every sequence, [kv_len[b], heads, head_dim], out of cache [pages, page_size, heads,
    head_dim]; zeros for a page id outside the cache."""
    pages, size = cache.shape[:2]
    found = []
    for b, L in enumerate(kv_len):
        x = np.zeros((int(L),) + cache.shape[2:], cache.dtype)
        for j in range(int(L)):
            page = int(table[b, j // size])
            if 0 <= page < pages:
                x[j] = cache[page, j % size]
        found.append(x)
    return found


def tolerance(out, lse, spread, reach, head_dim, keys, weight_eps, out_eps):
    """(largest error of out, of lse) of a computation that forms scores, weights and sums in fp32.

    A score is a sum of head_dim products: off by at most (head_dim + 4) 2^-24 reach (the sum's roundings, the
    scale's and the base's); the maximum's is common to a row's weights and its sum. exp is off by at most 4 * 2^-24
    and the argument's error, so a weight by d = 2 (head_dim + 4) 2^-24 reach + 2^-21 relative, and by weight_eps
    where it is rounded before it multiplies a value. Sums of `keys` terms in fp32 add (keys + 4) 2^-24, in
    numerator and denominator. The result's own rounding: out_eps of it."""
    d = 2 * (head_dim + 4) * 2.0 ** -24 * reach + 2.0 ** -21
    s = (keys + 4) * 2.0 ** -24
    e = (2 * d + 2 * s + weight_eps)[..., None] * spread
    finite = np.where(np.isfinite(lse), np.abs(lse), 0)
    return e + out_eps * (np.abs(out) + e) + 1e-30, d + s + 2.0 ** -22 * (1 + finite)
