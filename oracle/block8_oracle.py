"""Block-scaled E4M3 matrices, plain and slow in fp64 (numpy): the definition that
include/emeans.h states, sharing no code with the CUDA path."""

from __future__ import annotations

import numpy as np

BLOCK = 128
MIN_EXP, MAX_EXP = -117, 119

# The 256 E4M3 values (4 exponent bits of bias 7, 3 mantissa bits, no infinities, NaN
# where all seven bits are set).
_MAG = np.array([(m / 8.0) * 2.0 ** -6 if e == 0 else (1 + m / 8.0) * 2.0 ** (e - 7)
                 for e in range(16) for m in range(8)])
_MAG[127] = np.nan
E4M3 = np.concatenate([_MAG, -_MAG])
_GRID = _MAG[:127]


def blocks(d):
    return -(-d // BLOCK)


def exponent(a):
    """The block exponent for a largest magnitude a (Python float)."""
    if a == 0.0:
        return 0
    e = MIN_EXP
    while e < MAX_EXP and a > 448.0 * 2.0 ** e:
        e += 1
    return e


def nearest_code(v):
    """E4M3 code of |v| <= 448 by a search of the grid, ties to the even code."""
    if np.isnan(v):
        return 127
    a = abs(v)
    i = int(np.searchsorted(_GRID, a))
    if i > 126:
        i = 126
    if i > 0:
        lo, hi = _GRID[i - 1], _GRID[i]
        if a - lo < hi - a or (a - lo == hi - a and (i - 1) % 2 == 0):
            i -= 1
    return i | (128 if np.signbit(v) else 0)


def quantise(x):
    """(codes uint8 n x d, exponents int n x blocks) of the rows of x (fp64)."""
    n, d = x.shape
    codes = np.zeros((n, d), dtype=np.uint8)
    exps = np.zeros((n, blocks(d)), dtype=np.int64)
    mid = (_GRID[:-1] + _GRID[1:]) / 2
    for b in range(blocks(d)):
        v = x[:, b * BLOCK:(b + 1) * BLOCK]
        fin = np.isfinite(v)
        a = np.where(fin, np.abs(v), 0.0).max(axis=1)
        exps[:, b] = [exponent(float(t)) for t in a]
        s = np.where(fin, v, 0.0) / 2.0 ** exps[:, b, None].astype(np.float64)
        m = np.minimum(np.abs(s), 448.0)
        i = np.searchsorted(mid, m, side="left")  # midpoints below |v|
        tie = (i < len(mid)) & (m == mid[np.minimum(i, len(mid) - 1)])
        i = i + (tie & (i % 2 == 1))
        c = i.astype(np.uint8) | np.where(np.signbit(s), 128, 0).astype(np.uint8)
        codes[:, b * BLOCK:(b + 1) * BLOCK] = np.where(fin, c, 127)
    return codes, exps


def values(codes, exps):
    """fp64 values of codes with their exponents."""
    d = codes.shape[1]
    return E4M3[codes] * np.repeat(2.0 ** exps.astype(np.float64), BLOCK, axis=1)[:, :d]


def held(x):
    return values(*quantise(np.asarray(x, dtype=np.float64)))


def scale_at(row, block, d):
    groups = -(-blocks(d) // 4)
    return ((((row // 128) * groups + block // 4) * 32 + row % 32) * 4 + (row // 32) % 4) * 4 + block % 4


def exponents_of(scales, rows, d):
    """Exponents (len(rows) x blocks) of the given rows in an ordered scale buffer."""
    r = np.asarray(rows)[:, None]
    return scales[scale_at(r, np.arange(blocks(d))[None, :], d)].astype(np.int64) - 127
