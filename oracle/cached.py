"""fp64 reference of the paged key-value cache and of the attention over it, written from the
definitions, with Python's whole numbers and rationals where a rounding decides.

A token's head x, top = max |x|:
    e4m3:  s = the smallest power of two, at least 2^-126, with top <= 448 s;  code = x / s rounded
           to e4m3 (nearest, ties to even)
    int8:  s = top / 127 (fp32);  code = x * 127 / top rounded to a whole number (ties to even)
A head of zeros has scale 0, one with an infinity or NaN scale NaN and codes 0.

Position p of sequence b is in page table[b][p // page] at p % page; the rows start[b] ..
start[b + 1] of a call are the sequence's last positions before lens[b].
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def e4m3_values():
    """The 256 values of e4m3 (NaN where the code is one)."""
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c & 128, -v, v)


def round_half_even(x: Fraction) -> int:
    return round(x)  # Python rounds rationals to even


def quantise_head(x, kind):
    """x: finite or not, float64 [d] holding bf16 values -> (codes' values, scale as float)."""
    x = np.asarray(x, np.float64)
    if not np.isfinite(x).all():
        return np.zeros_like(x), math.nan
    top = np.abs(x).max()
    if top == 0:
        return np.zeros_like(x), 0.0
    if kind == "int8":
        t = Fraction(float(top))
        codes = [round_half_even(Fraction(float(v)) * 127 / t) for v in x]
        return np.array(codes, np.float64), float(np.float32(top) / np.float32(127))
    e = -126
    while top > 448 * 2.0 ** e:
        e += 1
    grid = np.unique(e4m3_values()[~np.isnan(e4m3_values())])
    y = x * 2.0 ** -e
    i = np.clip(np.searchsorted(grid, y), 1, len(grid) - 1)
    low, high = grid[i - 1], grid[i]
    # the nearer; the one with an even last place where both are as near
    even_low = np.round(low / (high - low)) % 2 == 0
    pick_low = (y - low < high - y) | ((y - low == high - y) & even_low)
    return np.where(pick_low, low, high), 2.0 ** e


def places(table, lens, start, page, n):
    """(sequence, position, page, slot) of every row with a token."""
    out = []
    for b in range(len(lens)):
        s0, s1 = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        for row in range(s0, s1):
            p = int(lens[b]) - (s1 - row)
            if 0 <= p and row < n:
                out.append((row, b, p, int(table[b][p // page]), p % page))
    return out


def attention(q, k, v, lens, start, window=None, span=False, scale=None, cap=0.0, slopes=None):
    """q [n, hq, d]; k / v: a list of [len, hkv, d] for every sequence.  Returns dict with o, lse
    and, for error bounds, "abs" = sum_j p_j |v_j| and "score" = the largest |scale q.k| terms
    sum_c |scale q_c k_c| of a row's visible keys."""
    n, hq, d = q.shape
    scale = 1 / math.sqrt(d) if scale is None else scale
    o, lse = np.zeros((n, hq, d)), np.full((hq, n), -np.inf)
    size, terms = np.zeros((n, hq, d)), np.zeros((hq, n))
    for b in range(len(lens)):
        s0, s1 = (b, b + 1) if start is None else (int(start[b]), int(start[b + 1]))
        length = int(lens[b])
        for row in range(s0, s1):
            p = length - (s1 - row)
            j = np.arange(length)
            see = (p - j >= 0) & (p - j < (math.inf if window is None else window))
            if span:
                see |= j >= length - (s1 - s0)
            if p < 0 or not see.any():
                continue
            for h in range(hq):
                g = h // (hq // k[b].shape[1])
                K, V = k[b][see, g], v[b][see, g]
                x = K @ q[row, h] * scale
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x - float(slopes[h]) * np.abs(p - j[see])
                top = x.max()
                w = np.exp(x - top)
                total = w.sum()
                o[row, h] = w @ V / total
                size[row, h] = w @ np.abs(V) / total
                lse[h, row] = top + math.log(total)
                terms[h, row] = (np.abs(K) @ np.abs(q[row, h])).max() * scale
    return {"o": o, "lse": lse, "abs": size, "terms": terms}
