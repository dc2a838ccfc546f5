"""Oracle of the unit's matrix products and 8-bit codes, in NumPy, from the
definitions; bf16 is carried as uint16 bit patterns, as in the other oracles.
"""

import numpy as np

from oracle import muon_oracle as M

widen, cast = M.widen, M.cast


def quantize(x, channel=None):
    """(codes int8, scales fp32) of the rows of an fp32 x [rows, cols]; channel:
    fp32, broadcast to x's shape.  Every reciprocal and product in fp32."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        if channel is not None:
            x = (x * np.asarray(channel, np.float32)).astype(np.float32)
        a = np.abs(x).max(-1, keepdims=True)           # NaN where a row has one
        one = np.float32(1)
        scale = (a * (one / np.float32(127))).astype(np.float32)
        factor = ((one / a).astype(np.float32) * np.float32(127)).astype(np.float32)
        codes = np.rint((x * factor).astype(np.float32))
    bad, tiny = ~np.isfinite(a), a < np.float32(2.0 ** -100)
    codes = np.where(bad | tiny, np.float32(0), codes)
    scale = np.where(bad, np.float32(np.nan), np.where(tiny, np.float32(0), scale))
    return codes.astype(np.int8), scale[..., 0].astype(np.float32)


def grouped(op, a, b, c, offsets, accumulate=False):
    """The product in 64 bits, and the sum of its terms' magnitudes (which its
    fp32 sums' error is relative to).  a, b, c: arrays of numbers; b [groups, ..]
    (nt, nn); c [groups, n, k] (tn).  Rows of no group keep c."""
    a, b, c = (np.asarray(x, np.float64) for x in (a, b, c))
    out = c.copy()
    size = np.zeros_like(out)
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if op == "tn":
            x, y = a[lo:hi].T, b[lo:hi]
            where = g
        else:
            x, y = a[lo:hi], b[g].T if op == "nt" else b[g]
            where = slice(lo, hi)
        out[where] = (out[where] if accumulate else 0) + x @ y
        size[where] = np.abs(x) @ np.abs(y) + (np.abs(c[where]) if accumulate else 0)
    return out, size


def grouped_i8(op, a, sa, b, sb, c, offsets, accumulate=False):
    """The product of codes in fp32, as it is documented: the exact sum rounded
    to fp32, times the row's scale, times the column's."""
    out = np.array(c, np.float32)
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        y = b[g].astype(np.int64)
        s = (a[lo:hi].astype(np.int64) @ (y.T if op == "nt" else y)).astype(np.float32)
        with np.errstate(all="ignore"):
            s = (s * sa[lo:hi, None]).astype(np.float32)
            if sb is not None:
                s = (s * sb[g][None, :]).astype(np.float32)
        out[lo:hi] = (out[lo:hi] + s).astype(np.float32) if accumulate else s
    return out
