"""Oracle of the operators on a cache held in 8 bits: plain numpy in float64.

A sequence's cache is codes [Hkv, cap, d] (bytes, e4m3) with scales [Hkv,
cap / 64]; an element is scale * value(code).  The functions work on one
sequence at a time and share no code with the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 64


def _decode(c: int) -> float:
    sign = -1.0 if c & 0x80 else 1.0
    e, m = (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    return sign * (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))


VALUES = np.array([_decode(c) for c in range(256)])  # by code
_POS = VALUES[:127]                                  # 0 .. 448, ascending with the code
_MID = (_POS[:-1] + _POS[1:]) / 2                    # a tie goes to the even code


def encode(x) -> np.ndarray:
    """The e4m3 code nearest to each value, ties to the even code; beyond
    +-448 the largest code, NaN the NaN code (its sign is not specified)."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    lo = np.searchsorted(_MID, a, side="left")    # codes whose upper midpoint is < a are passed
    hi = np.searchsorted(_MID, a, side="right")
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi)).astype(np.uint8)  # lo < hi: a tie
    code = np.where(np.isnan(x), 127, code)
    return np.where(np.signbit(x) & ~np.isnan(x), code | 0x80, code).astype(np.uint8)


def scale_of(amax: float) -> float:
    """The smallest 2^e >= 2^-126 with amax <= 448 * 2^e."""
    e = -126
    while amax > math.ldexp(448.0, e):
        e += 1
    return math.ldexp(1.0, e)


def append(codes, scales, x, length: int) -> None:
    """In place: the n new tokens x [n, Hkv, d] become tokens length-n .. length-1."""
    n, Hkv, _ = x.shape
    pos0 = length - n
    for blk in range(pos0 // BLOCK, (length - 1) // BLOCK + 1 if n else 0):
        lo, hi = max(pos0, blk * BLOCK), min(length, (blk + 1) * BLOCK)
        for h in range(Hkv):
            new = np.asarray(x[lo - pos0:hi - pos0, h], np.float64)
            fin = np.abs(new[np.isfinite(new)])
            s = scale_of(float(fin.max()) if fin.size else 0.0)
            if lo > blk * BLOCK:  # older tokens: the scale never shrinks
                old = float(scales[h, blk])
                old = old if 0 < old < math.inf else 0.0  # no scale: zeros
                s = max(s, old)
                if s != old:
                    part = codes[h, blk * BLOCK:lo]
                    codes[h, blk * BLOCK:lo] = encode(VALUES[part] * (old / s))
            codes[h, lo:hi] = encode(new / s)
            scales[h, blk] = s


def values(codes, scales) -> np.ndarray:
    """[Hkv, cap, d] as float64."""
    return VALUES[codes] * np.repeat(np.asarray(scales, np.float64), BLOCK, axis=-1)[..., None]


def index_scores(q, w, k):
    """q [H, d], w [H], k [n, d] -> (scores [n], sum_j |w_j| sum_c |q_jc k_c| [n])."""
    q, w, k = (np.asarray(t, np.float64) for t in (q, w, k))
    return np.maximum(k @ q.T, 0.0) @ w, np.abs(k) @ np.abs(q).T @ np.abs(w)


def attention(q, k, v, scale: float):
    """One KV head: q [R, d], k and v [n, d] -> (o [R, d], sum_t p_t |v_t| [R, d],
    max_t scale * sum_c |q_c k_c| [R]).  No token: zeros."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    if len(k) == 0:
        return np.zeros_like(q), np.zeros_like(q), np.zeros(len(q))
    z = scale * (q @ k.T)
    p = np.exp(z - z.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    return p @ v, p @ np.abs(v), scale * (np.abs(q) @ np.abs(k).T).max(1)
