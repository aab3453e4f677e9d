"""Paged K/V cache and attention over it, in float64 (TEST INFRASTRUCTURE, oracle).

Only the test suite may import this module.  The definitions written out:
position p of sequence b is row p % page of page table[b][p // page]; an 8-bit
row is its values over the smallest power of two that brings the largest
magnitude to 448 or less, rounded to the e4m3 grid (3 mantissa bits, normal
from 2^-6 on, the grid even below that); attention is softmax attention under
the mask "key j is one of the sequence's and, in causal order, not after the
query's own position".
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

E_MIN, E_MAX, E_BIAS, E_NAN = -100, 7, 127, 255


def e4m3_round(y: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (ties to even), saturating at +-448."""
    y = np.clip(np.asarray(y, dtype=np.float64), -448.0, 448.0)
    _, n = np.frexp(np.abs(y))                        # |y| = f 2^n, f in [1/2, 1)
    step = np.ldexp(1.0, np.maximum(n - 1, -6) - 3)
    return np.clip(np.round(y / step) * step, -448.0, 448.0)


def quantise_rows(x: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """Rows [..., D] -> (e4m3 values [..., D], exponent bytes [...])."""
    x = np.asarray(x, dtype=np.float64)
    bad = np.isnan(x).any(axis=-1)
    x = np.where(bad[..., None], 0.0, x)
    a = np.abs(x).max(axis=-1)
    e = np.full(a.shape, E_MIN, dtype=np.int64)
    while True:                                       # the definition, one step at a time
        more = (a > 448.0 * np.ldexp(1.0, e)) & (e < E_MAX)
        if not more.any():
            break
        e = e + more
    y = e4m3_round(np.clip(x, -1e300, 1e300) / np.ldexp(1.0, e)[..., None])
    return y, np.where(bad, E_NAN, e + E_BIAS).astype(np.uint8)


def dequantise_rows(y: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """Values of stored rows: y 2^(byte - 127), NaN throughout for byte 255."""
    byte = np.asarray(byte)
    scale = np.where(byte == E_NAN, np.nan, np.ldexp(1.0, byte.astype(np.int64) - E_BIAS))
    return np.asarray(y, dtype=np.float64) * scale[..., None]


def places(lengths: Sequence[int], offsets: Optional[Sequence[int]], table, page: int
           ) -> List[Tuple[int, int]]:
    """(page, row in page) of every packed token."""
    out = []
    for b, n in enumerate(lengths):
        off = 0 if offsets is None else int(offsets[b])
        out += [(int(table[b][p // page]), p % page) for p in range(off, off + n)]
    return out


def cached_rows(cache: np.ndarray, table_row, n: int) -> np.ndarray:
    """First n positions of a sequence out of cache values [P, page, H, D]."""
    page = cache.shape[1]
    out = np.zeros((n,) + cache.shape[2:], dtype=np.float64)
    for p in range(n):
        out[p] = cache[int(table_row[p // page]), p % page]
    return out


def paged_attention(q: np.ndarray, k_cache: np.ndarray, v_cache: np.ndarray,
                    lengths: Sequence[int], seq_lens: Sequence[int], table, causal: bool,
                    scale: float, heads: Optional[Sequence[int]] = None):
    """q [T, Hq, D] and cache values [P, page, Hkv, D] in float64.  Returns
    (out, weight, reach), each per row and head in `heads` (all): out the
    attention, weight = sum_j w_j |v_j| (what relative errors of the weights
    multiply) and reach = max_j scale sum_d |q_d k_jd| (what relative errors
    of the scores multiply, [T, Hq, 1])."""
    T, Hq, D = q.shape
    G = Hq // k_cache.shape[2]
    out, weight = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    reach = np.zeros((T, Hq, 1))
    t0 = 0
    for b, (lq, lk) in enumerate(zip(lengths, seq_lens)):
        k, v = cached_rows(k_cache, table[b], lk), cached_rows(v_cache, table[b], lk)
        i, j = np.arange(lq)[:, None], np.arange(lk)[None, :]
        allowed = (j <= lk - lq + i) if causal else np.ones((lq, lk), dtype=bool)
        for h in (range(Hq) if heads is None else heads):
            qh, kh, vh = q[t0:t0 + lq, h], k[:, h // G], v[:, h // G]
            s = np.where(allowed, (qh @ kh.T) * scale, -np.inf)
            top = s.max(axis=1, keepdims=True, initial=-np.inf)
            w = np.where(allowed, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
            den = w.sum(axis=1, keepdims=True)
            w = np.where(den > 0, w / np.where(den > 0, den, 1.0), 0.0)
            out[t0:t0 + lq, h] = w @ vh
            weight[t0:t0 + lq, h] = w @ np.abs(vh)
            size = np.where(allowed, (np.abs(qh) @ np.abs(kh).T) * abs(scale), 0.0)
            reach[t0:t0 + lq, h, 0] = size.max(axis=1, initial=0.0)
        t0 += lq
    return out, weight, reach
