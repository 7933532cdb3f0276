"""CPU reference of the 4-bit weights with group scales (NumPy, float64); test
infrastructure only, shares no code with the library.

A group (32 columns of a row) has the scale 2^e, e the smallest integer in
[-125, 125] with max|a| <= 7 * 2^e (e = 0 for zeros, NaN for a group that holds
one or an infinity); an element becomes the nearest e2m1 value of a / 2^e,
halves to the even code, 6 from 5 on.
"""
from __future__ import annotations

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
NAN_BYTE = 255


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest code 0..15 of each value by its distances to the two
    neighbours; bit 3 is the sign."""
    a = np.minimum(np.abs(v), 6.0)
    hi = np.clip(np.searchsorted(GRID, a), 0, 7)
    lo = np.maximum(hi - 1, 0)
    up, down = GRID[hi] - a, a - GRID[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return (pick | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def quantise(a: np.ndarray):
    """(codes uint8 n x k, scale bytes int n x groups)."""
    a = np.asarray(a, dtype=np.float64)
    n, k = a.shape
    groups = -(-k // 32)
    codes = np.zeros((n, k), dtype=np.uint8)
    scale = np.full((n, groups), 127, dtype=np.int64)
    for g in range(groups):
        blk = a[:, g * 32:(g + 1) * 32]
        bad = ~np.isfinite(blk).all(axis=1)
        top = np.abs(np.where(bad[:, None], 0.0, blk)).max(axis=1)
        e = np.full(n, -125)
        for _ in range(251):
            low = (7.0 * 2.0 ** e < top) & (e < 125)
            if not low.any():
                break
            e = np.where(low, e + 1, e)
        e = np.where(top == 0, 0, e)
        codes[:, g * 32:(g + 1) * 32] = np.where(bad[:, None], 0, encode(np.where(bad[:, None], 0.0, blk) * 2.0 ** -e[:, None].astype(float)))
        scale[:, g] = np.where(bad, NAN_BYTE, e + 127)
    return codes, scale


def values(codes: np.ndarray, scale: np.ndarray) -> np.ndarray:
    k = codes.shape[1]
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.where(scale == NAN_BYTE, np.nan, 2.0 ** (scale - 127.0))
    return v * np.repeat(s, 32, axis=1)[:, :k]


def buffers(a: np.ndarray):
    """The two byte buffers of the storage format."""
    codes, scale = quantise(a)
    n, k = codes.shape
    steps, rows16 = -(-k // 128), -(-n // 16) * 16
    quads = -(-steps // 4)
    cb = np.zeros(rows16 // 16 * steps * 1024, dtype=np.uint8)
    for c in range(k):
        r = np.arange(n)
        at = (r // 16 * steps + c // 128) * 1024 + c % 32 // 8 * 256 + r % 16 * 16 + c % 128 // 32 * 4 + c % 8 // 2
        cb[at] |= codes[:, c] << (4 * (c % 2))
    sb = np.full(rows16 * (quads * 16 + 1), 127, dtype=np.uint8)
    r, g = np.meshgrid(np.arange(n), np.arange(scale.shape[1]), indexing="ij")
    sb[(g // 16 * rows16 + r) * 16 + g % 16] = scale
    # a group of zeros does not count for its row's largest; one of NaN neither
    top = np.zeros(n, dtype=np.int64)
    for i in range(scale.shape[1]):
        live = (np.asarray(a)[:, i * 32:(i + 1) * 32] != 0).any(axis=1) & (scale[:, i] != NAN_BYTE)
        top = np.where(live, np.maximum(top, scale[:, i]), top)
    sb[quads * rows16 * 16 + np.arange(n)] = np.where(top == 0, 127, top)
    return cb, sb
