"""8-bit pages of a caller's pool in fp64 numpy, written from their definition.

Bytes [n_pages, n_kv, 64 * (2 * d + 8)]: per page of 64 tokens and head the key
codes [64][d], the value codes [64][d] (each code + 128), the key scales [64]
and the value scales [64] (fp32). `decode` gives the pool of
oracle/paged_cache.py that they stand for, so its definitions of attention
apply.
"""
from __future__ import annotations

import numpy as np

PAGE = 64
LEAST = 2.0 ** -100


def quantise(x):
    """Rows [..., d] -> (codes [..., d], scales [...]), both fp64: codes are
    whole numbers, a row with a non-finite value has the scale NaN."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore"):
        top = np.abs(x).max(axis=-1)
        held = np.isfinite(top) & (top >= LEAST)
        ratio = np.where(held, top, 1.0)
        codes = np.where(held[..., None], np.rint(np.where(held[..., None], x, 0.0) * (127.0 / ratio[..., None])), 0.0)
        scales = np.where(held, top / 127.0, np.where(np.isfinite(top), 0.0, np.nan))
    return codes, scales


def parts(pool, d):
    """(key codes, value codes [n, h, 64, d], key scales, value scales [n, h, 64]) in fp64."""
    pool = np.ascontiguousarray(pool)
    n, h, _ = pool.shape
    codes = pool[..., : 2 * PAGE * d].reshape(n, h, 2, PAGE, d).astype(np.float64) - 128.0
    scales = np.ascontiguousarray(pool[..., 2 * PAGE * d:]).view(np.float32).reshape(n, h, 2, PAGE).astype(np.float64)
    return codes[:, :, 0], codes[:, :, 1], scales[:, :, 0], scales[:, :, 1]


def rounded(x, bits):
    """x to `bits` significant bits, halves to the even one."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def decode(pool, d, bits=None, whole=False):
    """The pool [n_pages, 2, n_kv, 64 * d] in fp64 that the bytes stand for; with
    `bits`, scales and products are rounded to so many significant bits, or (whole)
    products only, of a scale in two parts of that many (code * rest, rounded, is
    added to code * most)."""
    kc, vc, ks, vs = parts(pool, d)
    n, h = ks.shape[:2]

    def product(codes, scales):
        scales = scales[..., None]
        if bits is None:
            return codes * scales
        most = rounded(scales, bits)
        rest = rounded(codes * rounded(scales - most, bits), bits) if whole else 0.0
        return rounded(codes * most + rest, bits)
    with np.errstate(invalid="ignore"):
        k, v = product(kc, ks), product(vc, vs)
    return np.stack([k.reshape(n, h, -1), v.transpose(0, 1, 3, 2).reshape(n, h, -1)], axis=1)


def encode(keys, values):
    """Rows [n_pages, n_kv, 64, d] of keys and values -> the bytes of a pool."""
    n, h, _, d = np.shape(keys)
    out = np.zeros((n, h, PAGE * (2 * d + 8)), dtype=np.uint8)
    for i, x in enumerate((keys, values)):
        codes, scales = quantise(x)
        out[..., i * PAGE * d:(i + 1) * PAGE * d] = (codes + 128).astype(np.uint8).reshape(n, h, -1)
        at = 2 * PAGE * d + i * 4 * PAGE
        out[..., at:at + 4 * PAGE] = scales.astype(np.float32).view(np.uint8).reshape(n, h, -1)
    return out
