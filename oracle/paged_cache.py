"""Paged-cache operators in fp64 numpy, written from their definitions.

A pool is [n_pages, 2, n_kv, 64 * d]: per page of 64 tokens the keys
[n_kv][64][d], then the values transposed [n_kv][d][64]. Sequence i has the
new tokens q_start[i] .. q_start[i+1]-1 and kv_len[i] cached tokens, the new
ones last.
"""
from __future__ import annotations

import numpy as np

PAGE = 64


def rotate(x, positions, base: float):
    """Rotate-half rotation of [T, heads, d] rows at integer positions."""
    x = np.asarray(x, dtype=np.float64)
    if base == 0:
        return x.copy()
    d = x.shape[-1]
    theta = float(base) ** (-2.0 * np.arange(d // 2) / d)
    angle = np.asarray(positions, dtype=np.float64)[:, None] * theta
    c, s = np.cos(angle)[:, None, :], np.sin(angle)[:, None, :]
    a, b = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def places(q_start, kv_len):
    """Per new token of every sequence: (token, sequence, cache position)."""
    out = []
    for i in range(len(kv_len)):
        n = int(q_start[i + 1]) - int(q_start[i])
        for j in range(n):
            out.append((int(q_start[i]) + j, i, int(kv_len[i]) - n + j))
    return out


def append(pool, k, v, q_start, kv_len, table, base, positions=None, q=None):
    """(new pool, rotated queries): tokens without a page, or before their
    cache, leave the pool alone; rows of no sequence leave q alone."""
    pool = np.array(pool, dtype=np.float64)
    n_pages, _, n_kv, width = pool.shape
    d = width // PAGE
    q_out = None if q is None else np.array(q, dtype=np.float64)
    for t, i, pos in places(q_start, kv_len):
        if pos < 0:
            continue
        at = [pos if positions is None else int(positions[t])]
        if q is not None:
            q_out[t] = rotate(np.asarray(q)[t:t + 1], at, base)[0]
        page = int(table[i][pos // PAGE])
        if not 0 <= page < n_pages:
            continue
        s = pos % PAGE
        pool[page, 0].reshape(n_kv, PAGE, d)[:, s] = rotate(np.asarray(k)[t:t + 1], at, base)[0]
        pool[page, 1].reshape(n_kv, d, PAGE)[:, :, s] = np.asarray(v)[t]
    return pool, q_out


def cached(pool, table, count, d):
    """Keys and values [count, n_kv, d] of the first `count` tokens, and which
    of them have a page."""
    pool = np.asarray(pool)
    n_pages, _, n_kv, _ = pool.shape
    k = np.zeros((count, n_kv, d))
    v = np.zeros((count, n_kv, d))
    there = np.zeros(count, dtype=bool)
    for g in range((count + PAGE - 1) // PAGE):
        page = int(table[g])
        lo, hi = g * PAGE, min(count, (g + 1) * PAGE)
        if not 0 <= page < n_pages:
            continue
        k[lo:hi] = pool[page, 0].reshape(n_kv, PAGE, d)[:, : hi - lo].transpose(1, 0, 2)
        v[lo:hi] = pool[page, 1].reshape(n_kv, d, PAGE)[:, :, : hi - lo].transpose(2, 0, 1)
        there[lo:hi] = True
    return k, v, there


def row(q, k, v, scale):
    """One query [d] over the keys it sees [n, d]: (output, sum of w|v|,
    largest scale * sum |q||k|); zeros when it sees none."""
    if len(k) == 0:
        z = np.zeros(v.shape[-1])
        return z, z, 0.0
    s = k @ q * scale
    w = np.exp(s - s.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale)


def attention(q, pool, q_start, kv_len, table, scale, window=0, sinks=0, causal=True, prefix_table=None, prefix_len=0):
    """(out [T, heads, d], sum of w|v| of the same shape, score sizes [T,
    heads], rows [T] that belong to a sequence)."""
    q = np.asarray(q, dtype=np.float64)
    T, heads, d = q.shape
    n_kv = np.asarray(pool).shape[2]
    group = heads // n_kv
    out, mass, size = np.zeros_like(q), np.zeros_like(q), np.zeros((T, heads))
    owned = np.zeros(T, dtype=bool)
    pk, pv, pthere = cached(pool, prefix_table, prefix_len, d) if prefix_len else (None, None, None)
    own = {}
    for t, i, pos in places(q_start, kv_len):
        owned[t] = True
        n = int(kv_len[i])
        if i not in own:
            own = {i: cached(pool, table[i], n, d)}
        k, v, there = own[i]
        key = np.arange(n)
        see = there & ((key <= pos) if causal else np.ones(n, dtype=bool))
        if window > 0:
            see &= (key > pos - window) | (key < sinks)
        k, v = k[see], v[see]
        if prefix_len:
            psee = pthere & ((np.arange(prefix_len) <= prefix_len + pos) if causal else np.ones(prefix_len, dtype=bool))
            k, v = np.concatenate([pk[psee], k]), np.concatenate([pv[psee], v])
        for h in range(heads):
            out[t, h], mass[t, h], size[t, h] = row(q[t, h], k[:, h // group], v[:, h // group], scale)
    return out, mass, size, owned
