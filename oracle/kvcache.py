"""Float64 oracle of the 8-bit paged key/value cache: append, read, attention.

Plain numpy from the definitions, a token and a head at a time where the definition is; shares no code with
the library. Layout as include/kq.h: codes k [pages, kv_heads, page, dim], v [pages, kv_heads, page / 16, dim, 16],
scales [pages, kv_heads] float32.
"""
from __future__ import annotations

from dataclasses import dataclass

import numpy as np

SCALE_FLOOR = np.float32(2.0 ** -100)


@dataclass
class Cache:
    k: np.ndarray
    v: np.ndarray
    k_scale: np.ndarray
    v_scale: np.ndarray

    @property
    def page(self) -> int:
        return self.k.shape[2]

    @classmethod
    def zeros(cls, pages, page, kv_heads, dim):
        return cls(np.zeros((pages, kv_heads, page, dim), np.int8), np.zeros((pages, kv_heads, page // 16, dim, 16), np.int8),
                   np.zeros((pages, kv_heads), np.float32), np.zeros((pages, kv_heads), np.float32))

    def copy(self):
        return Cache(self.k.copy(), self.v.copy(), self.k_scale.copy(), self.v_scale.copy())


def norm_rotate(x, weight, eps, rope_row, rot_dim, interleaved):
    """One head's entries x [dim] (float64): norm, then rotation by rope_row (cosines, then sines; None: none)."""
    y = np.asarray(x, np.float64).copy()
    if weight is not None:
        y = y / np.sqrt(np.mean(y * y) + np.float64(np.float32(eps))) * np.asarray(weight, np.float64)
    if rope_row is not None:
        h = rot_dim // 2
        c, s = np.asarray(rope_row[:h], np.float64), np.asarray(rope_row[h:rot_dim], np.float64)
        ia, ic = (np.arange(0, rot_dim, 2), np.arange(1, rot_dim, 2)) if interleaved else (np.arange(h), np.arange(h, rot_dim))
        a, b = y[ia].copy(), y[ic].copy()
        y[ia] = a * c - b * s
        y[ic] = b * c + a * s
    return y


def quantize_block(y, s_old):
    """New tokens' entries y [n, dim] of one block with scale so far s_old: (scale float32, codes int8, ratio for
    the codes already there)."""
    if not np.all(np.isfinite(y)) or np.isnan(s_old):
        return np.float32(np.nan), np.zeros(y.shape, np.int8), 1.0
    top = np.max(np.abs(y))
    s = max(np.float32(top / 127.0), SCALE_FLOOR) if top > 0 else np.float32(0.0)
    s = max(np.float32(s_old), s)
    if not np.isfinite(s):
        return np.float32(np.nan), np.zeros(y.shape, np.int8), 1.0
    if s == 0:
        return np.float32(0.0), np.zeros(y.shape, np.int8), 1.0
    codes = np.clip(np.rint(y / np.float64(s)), -127, 127).astype(np.int8)
    return s, codes, (np.float64(s_old) / np.float64(s) if s_old > 0 else 1.0)


def append(cache: Cache, table, lens, q_start, q, k, v, *, q_norm=None, k_norm=None, eps=1e-6, rope=None,
           interleaved=False):
    """Appends in place; returns the rotated queries [rows, heads, dim] float64 (rows of no sequence: NaN)."""
    page, kvh, dim = cache.page, k.shape[1], k.shape[2]
    rot = 0 if rope is None else rope.shape[1]
    out = np.full(q.shape, np.nan) if q is not None else None
    for b in range(len(lens)):
        r0, n, length = q_start[b], q_start[b + 1] - q_start[b], lens[b]
        first = length - n
        for i in range(n):
            p = first + i
            if q is not None and p >= 0 and (rope is None or p < len(rope)):
                for h in range(q.shape[1]):
                    out[r0 + i, h] = norm_rotate(q[r0 + i, h], q_norm, eps, None if rope is None else rope[p], rot, interleaved)
        if n == 0:
            continue
        start = max(first, 0)
        for p0 in range(start // page * page, length, page):
            lo, hi = max(start - p0, 0), min(page, length - p0)
            pg = table[b][p0 // page]
            if not 0 <= pg < cache.k.shape[0]:
                continue
            for h in range(kvh):
                ky = np.stack([norm_rotate(k[r0 + p0 + t - first, h], k_norm, eps,
                                           None if rope is None else (rope[p0 + t] if p0 + t < len(rope) else
                                                                      np.full(rot, np.nan)), rot, interleaved)
                               for t in range(lo, hi)])
                vy = np.asarray(v[r0 + p0 + lo - first:r0 + p0 + hi - first, h], np.float64)
                s, c, ratio = quantize_block(ky, cache.k_scale[pg, h] if lo else np.float32(0))
                cache.k[pg, h, :lo] = np.rint(cache.k[pg, h, :lo] * ratio)
                cache.k[pg, h, lo:hi] = c
                cache.k_scale[pg, h] = s
                s, c, ratio = quantize_block(vy, cache.v_scale[pg, h] if lo else np.float32(0))
                for t in range(lo):
                    cache.v[pg, h, t // 16, :, t % 16] = np.rint(cache.v[pg, h, t // 16, :, t % 16] * ratio)
                for t in range(lo, hi):
                    cache.v[pg, h, t // 16, :, t % 16] = c[t - lo]
                cache.v_scale[pg, h] = s
    return out


def tokens(cache: Cache, table_row, first, last):
    """Keys and values [last - first, kv_heads, dim] of positions first .. last - 1, float64 (a bad page: NaN)."""
    page, kvh, dim = cache.page, cache.k.shape[1], cache.k.shape[3]
    k, v = np.full((last - first, kvh, dim), np.nan), np.full((last - first, kvh, dim), np.nan)
    for p in range(first, last):
        pg, t = table_row[p // page], p % page
        if 0 <= pg < cache.k.shape[0]:
            k[p - first] = cache.k[pg, :, t].astype(np.float64) * cache.k_scale[pg].astype(np.float64)[:, None]
            v[p - first] = cache.v[pg, :, t // 16, :, t % 16].astype(np.float64) * cache.v_scale[pg].astype(np.float64)[:, None]
    return k, v


def attention(cache: Cache, table, lens, q_start, q, scale, window=0):
    """(out [rows, heads, dim], weight bound [rows, heads, dim], score bound [rows, heads], top [rows, heads]) in
    float64: the bounds are sum_t p_t |v_t|, scale * max_t sum_d |q_d k_td| and max_t p_t s_v,t (the block's scale),
    for tolerances. Rows of no sequence are NaN."""
    heads, dim = q.shape[1], q.shape[2]
    g = heads // cache.k.shape[1]
    out, vabs, smax = np.full(q.shape, np.nan), np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    top = np.full(q.shape[:2], np.nan)
    for b in range(len(lens)):
        r0, n, length = q_start[b], q_start[b + 1] - q_start[b], lens[b]
        if n == 0:
            continue
        low = max(0, length - n + 1 - window) if window else 0
        k, v = tokens(cache, table[b], low, length) if length > low else (None, None)
        pg = np.array([table[b][p // cache.page] for p in range(low, length)], np.int64)
        sv = cache.v_scale[np.where((pg >= 0) & (pg < len(cache.v_scale)), pg, 0)].astype(np.float64)
        for i in range(n):
            p = length - n + i
            a = max(low, p + 1 - window) if window else 0
            if p < 0:
                out[r0 + i], vabs[r0 + i], smax[r0 + i], top[r0 + i] = 0.0, 0.0, 0.0, 0.0
                continue
            for h in range(heads):
                kk, vv = k[a - low:p + 1 - low, h // g], v[a - low:p + 1 - low, h // g]
                qq = np.asarray(q[r0 + i, h], np.float64)
                e = (kk @ qq) * scale
                w = np.exp(e - np.max(e))
                w = w / np.sum(w)
                out[r0 + i, h], vabs[r0 + i, h] = w @ vv, w @ np.abs(vv)
                smax[r0 + i, h] = np.max(np.abs(kk) @ np.abs(qq)) * scale
                top[r0 + i, h] = np.max(w * sv[a - low:p + 1 - low, h // g])
    return out, vabs, smax, top
