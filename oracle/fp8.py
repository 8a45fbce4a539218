"""8-bit numbers with block scales: float64 CPU oracle.

TEST INFRASTRUCTURE ONLY -- imported by ``tests/``, never by the product path.
It shares no code with the HIP library.

* ``e4m3_round``: the nearest e4m3 value (four significant bits, multiples of
  2^-9, largest 448), ties to even.
* ``e4m3_bytes`` / ``e4m3_values``: values to codes and back.
* ``scale_bytes``: the E8M0 byte of a block from its largest magnitude.
* ``fp8_quantize``: rows in blocks of 128, or 128 x 128 tiles.
* ``fp8_values``: what codes and scales stand for.
"""
from __future__ import annotations

import numpy as np

__all__ = ["e4m3_round", "e4m3_bytes", "e4m3_values", "scale_bytes", "fp8_quantize", "fp8_values"]

BLOCK = 128


def e4m3_values(codes: np.ndarray) -> np.ndarray:
    """float64 values of e4m3 bytes: sign, four exponent bits (bias 7), three mantissa bits; 0x7F and 0xFF are NaN."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    e, m = c >> 3 & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (np.maximum(e, 1) - 10.0))
    v = np.where((c & 0x7F) == 0x7F, np.nan, v)
    return np.where(c & 0x80, -v, v)


_GRID = e4m3_values(np.arange(127))          # the values >= 0, ascending


def e4m3_bytes(x: np.ndarray) -> np.ndarray:
    """Nearest code by search in the table of values; |x| <= 448; of two equally near ones the even code."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x)
    hi = np.clip(np.searchsorted(_GRID, a), 1, 126)
    lo = hi - 1
    d_lo, d_hi = a - _GRID[lo], _GRID[hi] - a
    c = np.where(d_lo < d_hi, lo, np.where(d_hi < d_lo, hi, np.where(lo % 2 == 0, lo, hi)))
    return (c | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def e4m3_round(x: np.ndarray) -> np.ndarray:
    return e4m3_values(e4m3_bytes(x))


def scale_bytes(top: np.ndarray) -> np.ndarray:
    """The smallest byte b >= 27 with top <= 448 * 2^(b - 127); 255 for NaN and infinity."""
    top = np.asarray(top, dtype=np.float64)
    out = np.full(top.shape, 255, dtype=np.int64)
    for i in np.ndindex(top.shape):
        if np.isfinite(top[i]):
            b = 27
            while top[i] > 448.0 * 2.0 ** (b - 127):
                b += 1
            out[i] = b
    return out.astype(np.uint8)


def fp8_quantize(x: np.ndarray, tiles: bool = False):
    """(codes (rows, whole blocks), scale bytes) of float64 values."""
    rows, cols = x.shape
    nb, rt = -(-cols // BLOCK), -(-rows // BLOCK)
    full = np.zeros((rt * BLOCK, nb * BLOCK))
    full[:rows, :cols] = x
    blocks = full.reshape(rt * BLOCK, nb, BLOCK)
    top = np.abs(blocks).max(2)
    top = np.where(np.isnan(blocks).any(2), np.nan, top)
    if tiles:
        top = top.reshape(rt, BLOCK, nb).max(1)
    b = scale_bytes(top)
    each = np.repeat(b, BLOCK, 0) if tiles else b
    fine = each != 255
    with np.errstate(invalid="ignore", over="ignore"):
        v = blocks / 2.0 ** (each.astype(np.float64) - 127)[:, :, None]
    codes = e4m3_bytes(np.where(fine[:, :, None], v, 0.0))
    codes = np.where(fine[:, :, None], codes, 0x7F).astype(np.uint8).reshape(rt * BLOCK, nb * BLOCK)
    return codes[:rows], b if tiles else b[:rows]


def fp8_values(codes: np.ndarray, b: np.ndarray, tiles: bool = False) -> np.ndarray:
    s = np.where(b == 255, np.nan, 2.0 ** (b.astype(np.float64) - 127))
    s = np.repeat(s, BLOCK, 1)
    if tiles:
        s = np.repeat(s, BLOCK, 0)[:codes.shape[0]]
    return e4m3_values(codes) * s
