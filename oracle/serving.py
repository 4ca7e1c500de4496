"""Serving operators in float64 (oracle; test infrastructure only): causal attention of packed prompts, rows of a paged
key/value cache in bf16 or e4m3, attention of one new token per sequence.

e4m3 (one sign, four exponent bits of bias 7, three fraction bits, no infinities, S.1111.111 = NaN) is computed from its
bits; a row x is held as round(x / 2^e) with the smallest e in [-100, 120] that has max|x| <= 448 * 2^e. Each attention
returns, beside its result, sum_j p_j |v_j|: what a relative error of the weights is multiplied with.
"""
from __future__ import annotations

import numpy as np

EXP_MIN, EXP_MAX, BIAS, TOP = -100, 120, 127, 448.0


def e4m3_value(byte):
    """float64 values of e4m3 bytes."""
    b = np.asarray(byte, dtype=np.int64)
    s, e, m = np.where(b & 128, -1.0, 1.0), (b >> 3) & 15, b & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9.0)
    return np.where((b & 127) == 127, np.nan, s * v)


def e4m3_byte(x):
    """The e4m3 byte nearest to each x (ties to the even one), 448 for what is larger, NaN for NaN."""
    x = np.asarray(x, dtype=np.float64)
    grid = e4m3_value(np.arange(127))                       # ascending: 0 .. 448
    a = np.minimum(np.abs(x), TOP)
    hi = np.clip(np.searchsorted(grid, np.where(np.isnan(a), 0.0, a)), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    b = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    return np.where(np.isnan(x), 127, b | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def row_exponent(x):
    """e of each row (last axis), NaNs apart."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    a = np.max(np.where(np.isnan(a), 0.0, a), axis=-1)
    e = np.full(a.shape, EXP_MIN, dtype=np.int64)
    for cand in range(EXP_MIN, EXP_MAX):
        e += (a > TOP * 2.0 ** cand) & (e == cand)
    return e


def quantise(x):
    """(bytes, exponent bytes) of the rows of x."""
    e = row_exponent(x)
    with np.errstate(over="ignore"):
        return e4m3_byte(np.asarray(x, dtype=np.float64) * 2.0 ** -e[..., None].astype(np.float64)), \
            (e + BIAS).astype(np.uint8)


def stored_value(byte, exp):
    return e4m3_value(byte) * 2.0 ** (np.asarray(exp, dtype=np.float64) - BIAS)[..., None]


def attend(q, k, v, scale, mask):
    """(result, sum p |v|) of q [n, D] over k, v [m, D] where mask [n, m]; zeros for a row that sees nothing."""
    with np.errstate(invalid="ignore"):
        s = (q @ k.T) * scale
    s = np.where(mask, s, -np.inf)
    top = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    p = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    l = p.sum(axis=1, keepdims=True)
    p = np.where(l > 0, p / np.where(l > 0, l, 1.0), 0.0)
    out, mag = np.zeros((len(q), v.shape[1])), np.zeros((len(q), v.shape[1]))
    seen = mask.any(axis=0)                                 # keys nobody sees may hold anything
    full = np.isfinite(v).all(axis=1) & seen
    out += p[:, full] @ v[full]
    mag += p[:, full] @ np.abs(v[full])
    for j in np.flatnonzero(seen & ~full):
        with np.errstate(invalid="ignore"):
            out += np.where(mask[:, j:j + 1], p[:, j:j + 1] * v[j], 0.0)
    return out, mag


def prompt_attention(q, k, v, lens, scale):
    """q [T, Hq, D], k, v [T, Hk, D] float64, packed prompts of ``lens``: (out, sum p |v|) [sum lens, Hq, D]."""
    total, (_, hq, d), hk = sum(lens), q.shape, k.shape[1]
    out, mag, t = np.zeros((total, hq, d)), np.zeros((total, hq, d)), 0
    for n in lens:
        mask = np.tril(np.ones((n, n), dtype=bool))
        for h in range(hq):
            c = h // (hq // hk)
            out[t:t + n, h], mag[t:t + n, h] = attend(q[t:t + n, h], k[t:t + n, c], v[t:t + n, c], scale, mask)
        t += n
    return out, mag


def sequence_rows(pages, table_row, n):
    """Rows 0 .. n - 1 [n, Hk, D] of a sequence from pages [n_pages, Hk, page_size, D] of float64 values."""
    size = pages.shape[2]
    return np.stack([pages[table_row[p // size], :, p % size] for p in range(n)]) if n else \
        np.zeros((0, pages.shape[1], pages.shape[3]))


def paged_attention(q, k_pages, v_pages, table, lens, scale):
    """q [B, Hq, D]; float64 pages [n_pages, Hk, page_size, D]: (out, sum p |v|) [B, Hq, D]."""
    b, hq, d = q.shape
    hk = k_pages.shape[1]
    out, mag = np.zeros((b, hq, d)), np.zeros((b, hq, d))
    for i in range(b):
        k, v = sequence_rows(k_pages, table[i], lens[i]), sequence_rows(v_pages, table[i], lens[i])
        for c in range(hk):
            rows = slice(c * (hq // hk), (c + 1) * (hq // hk))
            out[i, rows], mag[i, rows] = attend(q[i, rows], k[:, c], v[:, c], scale,
                                                np.ones((hq // hk, len(k)), dtype=bool))
    return out, mag
