"""CPU reference of the 8-bit block-scaled matrices (NumPy, float64); test
infrastructure only, shares no code with the library.

A block (128 x 128 or 1 x 128) has the scale 2^e, e the smallest integer
>= -127 with max|a| <= 448 * 2^e over its finite elements (e = 0 without a
non-zero one); an element becomes the nearest e4m3 value of a / 2^e, halves to
the even code, and the NaN code 0xFF if it is not finite.
"""
from __future__ import annotations

import numpy as np


def e4m3_table() -> np.ndarray:
    """Value of each code 0..255 (sign, 4 exponent bits of bias 7, 3 mantissa
    bits; 0x7F and 0xFF are NaN, there are no infinities)."""
    out = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if e == 15 and m == 7:
            v = np.nan
        out[c] = -v if c & 128 else v
    return out


def encode(v: np.ndarray) -> np.ndarray:
    """Nearest code of each value, |v| <= 448 or NaN, by comparing distances
    with the two neighbours in the table of non-negative codes."""
    grid = e4m3_table()[:127]
    a = np.abs(np.nan_to_num(v, nan=0.0))
    hi = np.clip(np.searchsorted(grid, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    pick = np.where(np.isnan(v), 127, pick)
    return (pick | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def quantise(a: np.ndarray, block_rows: int):
    """(codes uint8 rows x k, exponents int per row and step)."""
    a = np.asarray(a, dtype=np.float64)
    rows, k = a.shape
    steps = -(-k // 128)
    codes = np.zeros((rows, k), dtype=np.uint8)
    exps = np.zeros((rows, steps), dtype=np.int64)
    for r in range(0, rows, block_rows):
        for s in range(steps):
            blk = a[r:r + block_rows, s * 128:(s + 1) * 128]
            fin = np.abs(blk[np.isfinite(blk)])
            top = fin.max() if fin.size else 0.0
            e = 0
            if top > 0:
                e = -127
                if top > 448.0 * 2.0 ** -127:
                    e = int(np.floor(np.log2(top / 448.0))) - 1
                    while 448.0 * 2.0 ** e < top:
                        e += 1
                    e = max(e, -127)
            exps[r:r + block_rows, s] = e
            codes[r:r + block_rows, s * 128:(s + 1) * 128] = np.where(
                np.isfinite(blk), encode(np.where(np.isfinite(blk), blk, 0.0) * 2.0 ** -e), 0xFF)
    return codes, exps


def values(codes: np.ndarray, exps: np.ndarray) -> np.ndarray:
    k = codes.shape[1]
    return e4m3_table()[codes] * np.repeat(2.0 ** exps.astype(np.float64), 128, axis=1)[:, :k]


def buffers(codes: np.ndarray, exps: np.ndarray):
    """The two byte buffers of the storage format."""
    rows, k = codes.shape
    steps, rows16 = -(-k // 128), -(-rows // 16) * 16
    cb = np.zeros(rows16 // 16 * steps * 2048, dtype=np.uint8)
    sb = np.full(-(-steps // 4) * rows16 * 4, 127, dtype=np.uint8)
    r, c = np.meshgrid(np.arange(rows), np.arange(k), indexing="ij")
    at = ((r // 16) * steps + c // 128) * 2048 + (c % 128) // 64 * 1024 + (c % 64) // 16 * 256 + (r % 16) * 16 + c % 16
    cb[at] = codes
    r, s = np.meshgrid(np.arange(rows), np.arange(steps), indexing="ij")
    sb[((s // 4) * rows16 + r) * 4 + s % 4] = exps + 127
    return cb, sb
