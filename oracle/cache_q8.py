"""8-bit key/value cache: quantisation with a scale per block of tokens and head.

Test infrastructure (see ``oracle/__init__.py``). A cache operand is a pair
(codes [B, n_cap, Hkv, D], scale [B, ceil(n_cap / block), Hkv]) of float64 arrays; ``codes``
holds the numbers that the 8-bit codes stand for, so a value is ``codes * scale``.

Writing rows into a block gives it s' = max(s, 2^E): 2^E is the smallest power of two (2^-100
at least) with max |new x| <= qmax 2^E, and s the block's scale if rows before the write live
in it, else 0. New rows become nearest(x / s'); the older rows of the block, if s' > s,
nearest(codes * s / s'). Nearest is to the format's numbers, ties to the even code.
"""
import math

import numpy as np

LEAST_EXP = -100


def numbers(fmt):
    """The non-negative numbers of a format, ascending; the k-th has code k."""
    if fmt == "int8":
        return np.arange(128, dtype=np.float64)                  # 0 .. 127
    # e4m3: exponent field e, mantissa field m; e = 0 is subnormal; the last code is NaN
    out = [m / 8.0 * 2.0 ** -6 if e == 0 else (1.0 + m / 8.0) * 2.0 ** (e - 7) for e in range(16) for m in range(8)]
    return np.array(out[:-1], dtype=np.float64)                  # up to 448


def nearest(y, fmt):
    """Each y rounded to the nearest number of the format, ties to the even code, beyond the
    largest to the largest."""
    t = numbers(fmt)
    a = np.abs(y)
    hi = np.clip(np.searchsorted(t, a), 0, len(t) - 1)           # first number >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - t[lo], t[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0)) | (a >= t[-1])
    return np.copysign(np.where(up, t[hi], t[lo]), y)


def block_scale(amax, fmt):
    """Smallest power of two s >= 2^-100 with amax <= qmax * s."""
    qmax = float(numbers(fmt)[-1])
    e = LEAST_EXP
    if amax > 0:
        e = max(e, math.frexp(amax / qmax)[1] - 2)               # at or below the answer
        while amax > qmax * 2.0 ** e:
            e += 1
    return 2.0 ** e


def write(codes, scale, x, start, block, fmt):
    """Write rows x [T, Hkv, D] (finite) of one sequence at `start`: codes [n_cap, Hkv, D] and
    scale [n_blk, Hkv] are changed in place."""
    x = np.asarray(x, dtype=np.float64)
    end = start + x.shape[0]
    for blk in range(start // block, (end + block - 1) // block if x.shape[0] else 0):
        a, e = max(start, blk * block), min(end, (blk + 1) * block)
        for h in range(x.shape[1]):
            new = x[a - start:e - start, h]
            older = a > blk * block
            s = float(scale[blk, h]) if older else 0.0
            s2 = max(s, block_scale(float(np.abs(new).max()), fmt))
            if older and s2 > s:
                codes[blk * block:a, h] = nearest(codes[blk * block:a, h] * s / s2, fmt)
            codes[a:e, h] = nearest(new / s2, fmt)
            scale[blk, h] = s2


def read(codes, scale, positions, block):
    """Values of `positions` of one sequence; a position outside the cache gives zeros."""
    out = np.zeros((len(positions), *codes.shape[1:]))
    for r, p in enumerate(positions):
        if 0 <= p < codes.shape[0]:
            out[r] = codes[p] * scale[p // block][:, None]
    return out
