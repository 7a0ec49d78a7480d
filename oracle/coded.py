"""Block-coded 8-bit operands in fp64: E4M3 codes with one power-of-two scale
per block of 128 along K (activations: per token row; weights: per 128 rows).

Rule of a block with finite magnitude maximum amax: e = the smallest integer
with amax <= 448 * 2^e, at least -118, and 0 for amax = 0; each finite element
becomes the E4M3 value nearest to x * 2^-e (ties to the even mantissa), each
other element the NaN code; the block stands for code * 2^e.  With e = 120, the
largest exponent bf16 elements reach, magnitudes stop at 240: 256 * 2^120 is
past the finite range.  The maximum runs
over the finite elements only.
"""
import math

import numpy as np

from .quant import E4M3, encode

BLOCK = 128
MIN_EXPONENT = -118


def exponent(amax):
    """Smallest e >= MIN_EXPONENT with amax <= 448 * 2^e; 0 for amax = 0."""
    if amax == 0.0:
        return 0
    e = math.frexp(amax)[1] - 9          # amax < 2^(e + 9) = 512 * 2^e
    return max(MIN_EXPONENT, e if amax <= math.ldexp(448.0, e) else e + 1)


def code(x, tall):
    """(values of the codes [R, K] float64 with NaN for the NaN code, exponents
    [ceil(R / tall), ceil(K / 128)]) of x [R, K] in tall x 128 blocks."""
    x = np.asarray(x, np.float64)
    R, K = x.shape
    vals = np.empty((R, K))
    exps = np.empty((-(-R // tall), -(-K // BLOCK)), np.int64)
    for i in range(exps.shape[0]):
        for b in range(exps.shape[1]):
            at = (slice(i * tall, (i + 1) * tall), slice(b * BLOCK, (b + 1) * BLOCK))
            blk = x[at]
            fin = np.isfinite(blk)
            e = exponent(float(np.abs(np.where(fin, blk, 0.0)).max()))
            exps[i, b] = e
            v = np.where(fin, blk, 0.0) * 2.0 ** -e
            q = E4M3[encode(np.clip(v, -240.0, 240.0) if e == 120 else v)]
            vals[at] = np.where(fin, q, np.nan)
    return vals, exps


def values(vals, exps, tall):
    """The numbers a coding stands for, code * 2^e."""
    R, K = vals.shape
    f = np.repeat(np.repeat(2.0 ** exps.astype(np.float64), tall, axis=0)[:R], BLOCK, axis=1)[:, :K]
    return vals * f
