"""How far an orthogonalisation's result may be off its 64-bit value."""

import numpy as np

from oracle import muon_oracle as M


def rms(x):
    return np.sqrt((np.asarray(x, np.float64) ** 2).mean())


def check(got, want, off, dtype, what=""):
    """got against the 64-bit values `want` of a matrix with at least 40 rows
    and columns; off: what the imitation of the library's precision is off
    them (rms).

    bf16: the result is the rounding of a value that is `off` away, give or
    take.  The two are independent, so their squares add: sqrt(r^2 + off^2)
    with r the rms of rounding `want` itself.  `off` is a sum over the
    roundings of at least 40 * 41 / 2 operands, at the same places with other
    sums: other orders and scales of one matrix's rows and columns moved it by
    0.90 to 1.08 on the CPU (13 shapes, three spectra), so half as much again
    is allowed.  r is the rms of N roundings, and the result's are others.  An
    error that is uniform over a step has a square of mean 1/12 and standard
    deviation 0.075 steps^2, 0.9 of the mean (over the steps of one binade and
    the next much the same): the rms is spread by 0.45 / sqrt(N), the
    difference of two by 0.64 / sqrt(N), three of which are allowed.

    fp32: three times `off`, as other orders of the sums are most of it, half
    a step, and what the fp32 arithmetic of the last step adds.  Any entry: 16
    times `off` and four times that, at the scale of the larger of the rms and
    itself."""
    assert min(want.shape) >= 40
    size = rms(want)
    d = M.widen(got).astype(np.float64) - want
    if dtype == "bf16":
        r = rms(M.widen(M.cast(want.astype(np.float32), "bf16")) - want)
        most = np.sqrt(r ** 2 + (1.5 * off) ** 2) * (1 + 3 * 0.64 / np.sqrt(want.size))
        half, last = 2.0 ** -8, 0.0
    else:
        half, last = 2.0 ** -24, 18 * 2.0 ** -22 / np.sqrt(min(want.shape)) * size
        most = half * size + 3 * off + last
    print(f"[gpu]   {what} {want.shape}: off {rms(d) / size:.3e}, allowed {most / size:.3e}",
          flush=True)
    assert rms(d) <= most, (what, rms(d) / size, most / size)
    scale = np.maximum(np.abs(want), size) / size
    assert (np.abs(d) <= half * np.abs(want) + (16 * off + 4 * last) * scale).all(), what


def spectrum(rng, r, c, kind):
    """White, two strong directions over white noise, or singular values 1 / k."""
    if kind == "white":
        return rng.standard_normal((r, c))
    if kind == "low":
        return 0.1 * rng.standard_normal((r, c)) + \
            rng.standard_normal((r, 2)) @ rng.standard_normal((2, c))
    k = min(r, c)
    q, _ = np.linalg.qr(rng.standard_normal((r, k)))
    p, _ = np.linalg.qr(rng.standard_normal((c, k)))
    return (q / np.arange(1, k + 1)) @ p.T
