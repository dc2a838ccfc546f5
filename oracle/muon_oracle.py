"""Oracle of the Muon step: NumPy, float64 where the definition is, fp32 where
the library's contract rounds.  Test infrastructure only."""

from __future__ import annotations

import math

import numpy as np

from oracle import fsdp_oracle as O

POLY = (3.4445, -4.7750, 2.0315)


def matrices(shapes):
    """Parameters of two dimensions or more: (index, offset, rows, columns)."""
    out, at = [], 0
    for p, s in enumerate(shapes):
        n = int(np.prod(s))
        if len(s) >= 2:
            out.append((p, at, s[0], n // s[0]))
        at += n
    return out


def shard_map(po):
    """[T] -> place in the buffer [R*S]."""
    m = np.full(po.T, -1, np.int64)
    for r in range(po.R):
        for f0, s0, n in po.pieces(r):
            m[f0:f0 + n] = r * po.S + s0 + np.arange(n)
    return m


def chosen_mask(shapes, params):
    """[T]: whether an element belongs to a chosen parameter."""
    ends = np.cumsum([0] + [int(np.prod(s)) for s in shapes])
    mask = np.zeros(ends[-1], bool)
    for p in params:
        mask[ends[p]:ends[p + 1]] = True
    return mask


def widen(a):
    """fp32 values of fp32, or of bf16 bits."""
    return (a.astype(np.uint32) << 16).view(np.float32) if a.dtype == np.uint16 else a


def cast(a, dtype):
    return O.bf16_rne(a) if dtype == "bf16" else a.astype(np.float32)


def mean(grads):
    """fp32, in rank order, one division."""
    s = widen(grads[0]).copy()
    for g in grads[1:]:
        s = s + widen(g)
    return s / np.float32(len(grads))


def momentum(g, m, mu, nesterov):
    """One element-wise update from the averaged fp32 gradient."""
    gd = (1.0 - mu) * g.astype(np.float64)
    new = (mu * m.astype(np.float64) + gd).astype(np.float32)
    u = (gd + mu * new.astype(np.float64)).astype(np.float32) if nesterov else new
    return new, u


def scale_of(rows, cols, scale):
    if scale == "aspect":
        return np.sqrt(np.float64(max(1.0, rows / cols)))
    if scale == "rms":
        return 0.2 * np.sqrt(np.float64(max(rows, cols)))
    return 1.0


def apply(p, x, lr, wd, scale):
    return (p.astype(np.float64) * (1.0 - lr * wd) -
            (lr * scale) * x.astype(np.float64)).astype(np.float32)


def orthogonalize(u, steps=5, eps=1e-7, poly=POLY):
    """The definition, float64."""
    a, b, c = poly
    x = u.astype(np.float64)
    x = x / (np.sqrt((x * x).sum()) + eps)
    t = x.shape[0] > x.shape[1]
    x = x.T if t else x
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    return x.T if t else x


def plane_exponents(sigma, steps, poly):
    """The exponents q of the steps' results, whose planes hold X 2^-q: X's
    singular values are at most sigma before the first step and at most
    |a| s + |b| s^3 + |c| s^5 after one that began with at most s."""
    out = []
    for _ in range(steps):
        bound = sum(abs(k) * sigma ** p for k, p in zip(poly, (1, 3, 5)))
        out.append(max(min(math.frexp(bound)[1] - 1 if bound > 0 else -400, 0), -400))
        sigma = min(bound, 16.0)
    return out


def orthogonalize_rounded(u, steps=5, eps=1e-7, poly=POLY, split=False, diagonals=True,
                          low=True):
    """The definition with the library's documented precision: operands of
    11 bits (split: of 22) under power-of-two scales, fp32 sums, the residual
    of 14 bits (split: of 22) and the diagonals of A and B in fp32.  What it is off the definition by
    is what the kernels may be off by.  Without diagonals or low, those of A and
    B are in the planes, or the residual has 11 bits: what a kernel that lost
    them would compute."""
    f32 = np.float32

    def parts(x, s):
        hi = (x * f32(s)).astype(np.float16).astype(f32)
        lo = (x * f32(s) - hi).astype(np.float16)
        if not split:   # 5 bits of exponent and 2 of mantissa: fp16's upper byte, rounded
            b = lo.view(np.uint16)
            lo = ((b + 0x7f + ((b >> 8) & 1)) & 0xff00).astype(np.uint16).view(np.float16)
        lo = lo.astype(f32)
        return hi / f32(s), lo / f32(s)

    def prod(p, q):
        r = p[0] @ q[0]
        return r + (p[0] @ q[1] + p[1] @ q[0]) if split else r

    mass = float(np.sqrt((u.astype(np.float64) ** 2).sum()))
    norm = mass + eps
    e = math.frexp(mass)[1] - 1 if mass > 0 else 0
    f = math.ldexp(1.0, e) / norm if mass > 0 else 0.0
    exps = plane_exponents(mass / norm, steps, poly)
    x = (u.astype(np.float64) * 2.0 ** -e).astype(f32)
    t = x.shape[0] > x.shape[1]
    x = np.ascontiguousarray(x.T if t else x)
    for s in range(steps):
        if s == 0:
            scales = [f ** p * 2.0 ** -exps[0] for p in (1, 3, 5)]
        else:
            scales = [2.0 ** (p * exps[s - 1] - exps[s]) for p in (1, 3, 5)]
        a, b, c = [f32(k * z) for k, z in zip(poly, scales)]
        x = parts(x, 4096)
        if not low:
            x = (x[0], np.zeros_like(x[1]))
        g = prod(x, (x[0].T, x[1].T))
        d = np.diag(g).copy() if diagonals else np.zeros(len(g), f32)
        g = parts(g - np.diag(d), 1024)
        own = g[0] + g[1] if split else g[0]
        y = (b + c * (d[:, None] + d[None])) * own + c * prod(g, g)
        if diagonals:
            d = d * (b + c * d) + np.diag(y)
            np.fill_diagonal(y, 0)
        y = parts(y, 1024)
        x = (a + d)[:, None] * (x[0] + x[1]) + prod(y, x)
    x = (x.astype(np.float64) * 2.0 ** exps[-1]).astype(f32)
    return x.T if t else x
