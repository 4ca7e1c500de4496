"""The operators around a paged serving step in float64 (oracle; test infrastructure only): lengths, block tables and free
pages of sequences that grow and shrink, norms of heads with their rotation by position, rows held in 4 bits.

4-bit rows: groups of 16 elements; a scale byte is an fp16 value's exponent and first three fraction bits (no sign), the
scale nearest to max|x| / 6 of those up to 10240; an element is the e2m1 value nearest to x / scale. Ties go to the even code.
"""
from __future__ import annotations

import numpy as np

GROUP, NAN_BYTE, TOP_BYTE = 16, 0xFF, 0xE2
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def resize(by, lens, table, free, page_size):
    """(lens, table, free, cu_rows, positions, slots) after each sequence took by[b] tokens more: lists and arrays of the
    same shapes, one page after the other. free[0] counts the stack free[1:]."""
    lens, table, free = [int(x) for x in lens], np.array(table), [int(x) for x in free]
    pages = lambda n: -(-n // page_size)
    for b in reversed(range(len(lens))):
        for nth in reversed(range(pages(lens[b] + int(by[b])), pages(lens[b]))):
            free[0] += 1
            free[free[0]] = int(table[b, nth])
    cu, positions, slots = [0], [], []
    for b in range(len(lens)):
        n = int(by[b])
        for nth in range(pages(lens[b]), pages(lens[b] + n)):
            table[b, nth] = free[free[0]]
            free[0] -= 1
        for p in range(lens[b], lens[b] + n):
            positions.append(p)
            slots.append(int(table[b, p // page_size]) * page_size + p % page_size)
        lens[b] += n
        cu.append(len(positions))
    return lens, table, free, cu, positions, slots


def norm_rope(x, gain, eps, positions, freqs, neighbours):
    """(result, size of each element's pair before the rotation) of heads x [tokens, heads, D] float64; freqs: radians for
    one position of each pair."""
    y = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    if gain is not None:
        y = y * gain
    half, out, size = len(freqs), y.copy(), np.abs(y)
    if half:
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if neighbours else (slice(0, half), slice(half, 2 * half))
        w = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freqs, dtype=np.float64)
        out[..., a] = y[..., a] * np.cos(w) - y[..., b] * np.sin(w)
        out[..., b] = y[..., a] * np.sin(w) + y[..., b] * np.cos(w)
        size[..., a] = size[..., b] = np.hypot(y[..., a], y[..., b])
    return out, size


def scale_value(byte):
    """float64 values of scale bytes."""
    b = np.asarray(byte, dtype=np.int64)
    e, m = b >> 3, b & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 18.0), m * 2.0 ** -17.0)
    return np.where(e == 31, np.where(m, np.nan, np.inf), v)


def _nearest(x, grid):
    """The place in the ascending grid of the entry nearest to each x >= 0 (ties to the even place, the last for more)."""
    x = np.minimum(x, grid[-1])
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    dl, dh = x - grid[lo], grid[hi] - x
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def quantise(x):
    """(codes of 4 bits, scale bytes) of the rows of x; a group with a NaN or an infinity has byte 0xFF and codes of 0."""
    x = np.asarray(x, dtype=np.float64).reshape(*np.shape(x)[:-1], np.shape(x)[-1] // GROUP, GROUP)
    fin = np.isfinite(x).all(axis=-1)
    x = np.where(fin[..., None], x, 0.0)
    byte = _nearest(np.max(np.abs(x), axis=-1) / 6, scale_value(np.arange(TOP_BYTE + 1)))
    s = scale_value(byte)[..., None]
    code = _nearest(np.abs(x) / np.where(s > 0, s, 1.0), E2M1)
    code = np.where(s > 0, code + 8 * (x < 0), 0)
    return code.reshape(*x.shape[:-2], GROUP * x.shape[-2]).astype(np.uint8), np.where(fin, byte, NAN_BYTE).astype(np.uint8)


def pack(code):
    """Two codes a byte, the first in the low half."""
    return code[..., 0::2] | code[..., 1::2] << 4


def stored_value(packed, byte):
    """float64 values of packed rows."""
    code = np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], 2 * packed.shape[-1])
    v = np.where(code & 8, -1.0, 1.0) * E2M1[code & 7]
    with np.errstate(invalid="ignore"):
        return v * np.repeat(scale_value(byte), GROUP, axis=-1)
