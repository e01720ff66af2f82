"""Rotary positions, the paged e4m3 cache and attention over it, in float64 numpy.

Written from the definitions in include/moe_lora.h, one token, page or row at
a time, for the tests; the CUDA library shares no code with it.
"""
from __future__ import annotations

import numpy as np

E4M3_VALUES = np.array([(-1.0 if c & 0x80 else 1.0) * (
    (c & 7) * 2.0 ** -9 if (c >> 3) & 15 == 0 else (1 + (c & 7) / 8.0) * 2.0 ** (((c >> 3) & 15) - 7))
    for c in range(256)])
E4M3_VALUES[[0x7F, 0xFF]] = np.nan


def e4m3_encode(x):
    """Codes of float64 values: nearest, ties to the even code, magnitudes past
    448 give 448, NaN the NaN code."""
    x = np.asarray(x, dtype=np.float64)
    mags = E4M3_VALUES[:0x7F]
    a = np.minimum(np.abs(x), 448.0)
    nan = np.isnan(x)
    a = np.where(nan, 0.0, a)
    hi = np.clip(np.searchsorted(mags, a), 1, 0x7E)      # mags[hi - 1] < a <= mags[hi]
    lo = hi - 1
    up, down = mags[hi] - a, a - mags[lo]
    take = (up < down) | ((up == down) & (hi % 2 == 0))
    code = np.where(take, hi, lo).astype(np.uint8)
    code |= np.where(np.signbit(x), 0x80, 0).astype(np.uint8)
    return np.where(nan, np.uint8(0x7F), code)


def rotate(x, pos, freqs, mscale=1.0, interleaved=False, inverse=False):
    """x [H, D] of one token at position ``pos``."""
    y = np.array(x, dtype=np.float64)
    R = 2 * len(freqs)
    for i, f in enumerate(freqs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + R // 2)
        c, s = mscale * np.cos(pos * f), mscale * np.sin(pos * f)
        if inverse:
            s = -s
        u, w = x[:, a].astype(np.float64), x[:, b].astype(np.float64)
        y[:, a], y[:, b] = u * c - w * s, w * c + u * s
    return y


def page_scale(amax):
    """The smallest power of two, at least 2^-42, with amax <= 448 times it."""
    s = 2.0 ** -42
    while amax > 448.0 * s:
        s *= 2.0
    return s


def attend(q, k_codes, v_codes, k_scale, v_scale, block_table, seq_lens, cu_q, scale, window=0):
    """q [N, Hq, D]; codes [pages, Hkv, P, D] uint8.  Returns out, lse, and for
    error bounds sum_j p_j |v_j| [N, Hq, D] and the largest sum_d |q_d k_jd| *
    scale of a row [N, Hq]."""
    N, Hq, D = q.shape
    Hkv, P = k_codes.shape[1:3]
    out = np.zeros((N, Hq, D))
    lse = np.full((N, Hq), -np.inf)
    spread, size = np.zeros((N, Hq, D)), np.zeros((N, Hq))
    for b in range(len(seq_lens)):
        n = cu_q[b + 1] - cu_q[b]
        for t in range(n):
            i = seq_lens[b] - n + t
            js = [j for j in range(max(0, i - window + 1) if window else 0, i + 1)
                  if 0 <= block_table[b][j // P] < k_codes.shape[0]]
            if not js:
                continue
            pg = np.array([block_table[b][j // P] for j in js])
            off = np.array([j % P for j in js])
            for h in range(Hq):
                kv = h // (Hq // Hkv)
                k = E4M3_VALUES[k_codes[pg, kv, off]] * k_scale[pg, kv][:, None].astype(np.float64)
                v = E4M3_VALUES[v_codes[pg, kv, off]] * v_scale[pg, kv][:, None].astype(np.float64)
                row = q[cu_q[b] + t, h].astype(np.float64)
                s = scale * (k @ row)
                m = s.max()
                e = np.exp(s - m)
                r = cu_q[b] + t, h
                out[r] = (e / e.sum()) @ v
                lse[r] = m + np.log(e.sum())
                spread[r] = (e / e.sum()) @ np.abs(v)
                size[r] = scale * (np.abs(k) @ np.abs(row)).max()
    return out, lse, spread, size
