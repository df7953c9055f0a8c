"""Block-scaled fp8 in float64 (oracle side).

TEST INFRASTRUCTURE ONLY (see oracle/__init__.py).

A block (128 elements along the contraction axis, or a 128 x 128 tile) has the
scale 2^e, e the smallest integer >= -127 with max |a| <= 448 * 2^e; an
element's code is a / 2^e rounded to the nearest E4M3FN value, ties to the
even code.  A block with a value that is not finite has e = 0 and NaN codes.
"""

import math

import numpy as np

BLOCK = 128

# the 127 non-negative E4M3FN values in the order of their codes
GRID = np.array([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)][:127])


def exponent(amax):
    """The smallest e >= -127 with amax <= 448 * 2^e."""
    e = -127
    if amax > 0:
        e = max(-127, math.floor(math.log2(amax / 448.0)) - 2)
        while amax > 448.0 * 2.0 ** e:
            e += 1
    return e


def encode(v):
    """E4M3FN codes of finite v, |v| <= 448."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    i = np.clip(np.searchsorted(GRID, a, side="right") - 1, 0, 125)   # GRID[i] <= a
    lo, hi = GRID[i], GRID[i + 1]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 1))
    return (i + up).astype(np.uint8) | np.where(np.signbit(v), 0x80, 0).astype(np.uint8)


def decode(codes):
    c = np.asarray(codes)
    mag = np.concatenate([GRID, [np.nan]])[c & 0x7F]
    return np.where(c & 0x80, -mag, mag)


def _blocks(n):
    return -(-n // BLOCK)


def quantize(a, tile=False):
    """(codes rows x cols, scale bytes rows x blocks) of a (rows x cols)."""
    a = np.asarray(a, np.float64)
    rows, cols = a.shape
    codes = np.zeros((rows, cols), np.uint8)
    scales = np.zeros((rows, _blocks(cols)), np.uint8)
    step = BLOCK if tile else 1
    for r in range(0, rows, step):
        for b in range(_blocks(cols)):
            rs, cs = slice(r, r + step), slice(b * BLOCK, (b + 1) * BLOCK)
            blk = a[rs, cs]
            if not np.isfinite(blk).all():
                codes[rs, cs], scales[rs, b] = 0x7F, 127
                continue
            e = exponent(float(np.max(np.abs(blk))))
            codes[rs, cs] = encode(blk / 2.0 ** e)
            scales[rs, b] = e + 127
    return codes, scales


def dequantize(codes, scales):
    s = np.repeat(2.0 ** (scales.astype(np.float64) - 127), BLOCK, axis=1)
    return decode(codes) * s[:, :codes.shape[1]]


def seg_starts(offsets):
    """First column of each segment in a grouped transposed copy."""
    n = np.diff(offsets)
    return np.concatenate([[0], np.cumsum(-(-n // BLOCK) * BLOCK)])
