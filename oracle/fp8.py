"""The 8-bit KV cache row, from its definition, in float64.

A row x is stored as e4m3 codes and a byte b = e + 127, e the least integer
>= -126 with max|x| <= 448 * 2^e; code = the e4m3 value nearest to x * 2^-e, ties
to the even code.  A row with a NaN or an infinity: zeros and b = 255.
"""
import numpy as np

# value of every non-negative finite e4m3 code 0 .. 126: 4 exponent bits (bias 7), 3 fraction bits
VALUES = np.array([(c & 7) * 2.0 ** -9 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7) for c in range(127)])


def row_exponent(largest):
    """Least e >= -126 with largest <= 448 * 2^e (found by trying them all)."""
    for e in range(-126, 128):
        if largest <= 448 * 2.0 ** e:
            return e
    raise ValueError("not a bf16 magnitude")


def _nearest(y):
    """Codes of the e4m3 values nearest to y >= 0, ties to the even code."""
    hi = np.clip(np.searchsorted(VALUES, y), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = VALUES[hi] - y, y - VALUES[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))


def quantise(x):
    """x float64 [..., A] -> (codes uint8 [..., A], exponent bytes uint8 [...])."""
    x = np.asarray(x, np.float64)
    rows = x.reshape(-1, x.shape[-1])
    codes = np.zeros(rows.shape, np.uint8)
    exps = np.zeros(rows.shape[0], np.uint8)
    for i, row in enumerate(rows):
        if not np.isfinite(row).all():
            exps[i] = 255
            continue
        e = row_exponent(np.abs(row).max())
        code = _nearest(np.abs(row) * 2.0 ** -e)
        codes[i] = code | np.where(np.signbit(row), 128, 0)
        exps[i] = e + 127
    return codes.reshape(x.shape), exps.reshape(x.shape[:-1])


def values(codes, exps):
    """The float64 values that codes [..., A] and exponent bytes [...] stand for."""
    c = np.asarray(codes)
    if ((c & 127) == 127).any():
        raise ValueError("a stored code is a NaN pattern")
    v = np.where(c & 128, -1.0, 1.0) * VALUES[c & 127]
    e = np.asarray(exps).astype(np.int64)
    return np.where((e == 255)[..., None], np.nan, v * np.exp2((e - 127).astype(np.float64))[..., None])


def as_queried(q):
    """What attention takes finite query rows [..., A] (bf16 values) as: two e4m3
    terms, each nearest, of the row times the power of two that brings its largest
    magnitude into [128, 256) (at most 2^126)."""
    q = np.asarray(q, np.float64)
    largest = np.abs(q).max(-1, keepdims=True)
    shift = np.minimum(8 - np.frexp(largest)[1], 126)
    y = np.where(largest > 0, q * np.exp2(shift.astype(np.float64)), 0.0)
    hi = np.sign(y) * VALUES[_nearest(np.abs(y))]
    rest = y - hi
    return (hi + np.sign(rest) * VALUES[_nearest(np.abs(rest))]) * np.exp2(-shift.astype(np.float64))
