"""The orthogonalisation's documented precision, imitated on the CPU (no GPU):
its results are near the definition's for updates of every size beside eps."""

import numpy as np
import pytest

from oracle import muon_oracle as M
from tests import muon_check as C


@pytest.mark.parametrize("split", [False, True])
@pytest.mark.parametrize("shape", [(96, 160), (130, 61)])
def test_updates_far_below_eps(shape, split):
    """X = U / (|U|_F + eps) is small there and the steps nearly linear; the
    operands keep their bits all the same.  Each of the five steps rounds an
    entry's high part to 11 bits and its low part to 3 more (split: to 22),
    and adds the products' share, which |X|^2 makes small: below 5 * 2^-14
    (split: fp32 sums of a few terms, 5 * 4 * 2^-23) in all."""
    u = np.random.default_rng(1).standard_normal(shape).astype(np.float32)
    norm = np.linalg.norm(u.astype(np.float64))
    for ratio in (1e-2, 1e-4, 1e-6, 1e-8, 1e-9, 1e-20, 1e-35):
        want = M.orthogonalize(u, eps=norm / ratio)
        got = M.orthogonalize_rounded(u, eps=norm / ratio, split=split)
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off < (20 * 2.0 ** -23 if split else 5 * 2.0 ** -14), (ratio, off)


def test_exponents_of_the_planes():
    """None where eps does not matter; otherwise X's bound, step by step."""
    assert M.plane_exponents(1.0, 5, M.POLY) == [0] * 5
    assert M.plane_exponents(2.0 ** -40, 3, (4.0, 0.0, 0.0)) == [-38, -36, -34]
    assert M.plane_exponents(2.0 ** -3, 4, (4.0, 0.0, 0.0)) == [-1, 0, 0, 0]
    assert M.plane_exponents(1.0, 3, (0.25, 0.0, 0.0)) == [-2, -4, -6]
    assert M.plane_exponents(0.0, 2, M.POLY) == [-400] * 2


def test_steps_that_shrink_the_update():
    u = np.random.default_rng(2).standard_normal((40, 70)).astype(np.float32)
    for split in (False, True):
        want = M.orthogonalize(u, 16, poly=(0.25, 0.0, 0.0))
        got = M.orthogonalize_rounded(u, 16, poly=(0.25, 0.0, 0.0), split=split)
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off < 16 * (4 * 2.0 ** -23 if split else 2.0 ** -14), off
        assert (M.orthogonalize_rounded(u, 8, poly=(0.0, 1.0, 0.0), split=split) == 0).all()


SIDES = [(63, 64), (65, 191), (333, 100), (129, 129), (257, 255), (40, 1025), (320, 960)]


def rounded(u, dtype, **what):
    return M.cast(M.orthogonalize_rounded(u, split=dtype == "f32", **what).astype(np.float32),
                  dtype)


@pytest.mark.parametrize("r,c", SIDES)
def test_the_check_takes_results_of_the_documented_precision(r, c):
    """Rows and columns in another order and the matrix half as large again:
    the same value with other roundings."""
    for kind in ("white", "low", "steep"):
        rng = np.random.default_rng(r * 1000 + c)
        u = M.widen(M.cast((C.spectrum(rng, r, c, kind) * 1e-3).astype(np.float32), "bf16"))
        want = M.orthogonalize(u)
        p, q = rng.permutation(r), rng.permutation(c)
        for dtype in ("bf16", "f32"):
            off = C.rms(M.orthogonalize_rounded(u, split=dtype == "f32") - want)
            other = rounded(u[p][:, q] * np.float32(1.5), dtype)
            C.check(other, M.orthogonalize(u[p][:, q] * np.float32(1.5)), off, dtype, kind)


@pytest.mark.parametrize("r,c", SIDES)
def test_the_check_refuses_lost_diagonals_and_low_parts(r, c):
    """The diagonals of A and B rounded with their planes, and the residual a
    X in 11 bits, in the spectra where each matters."""
    for kind, lost, dtypes in (("white", "diagonals", ("bf16",)), ("low", "low", ("bf16", "f32"))):
        rng = np.random.default_rng(r * 1000 + c)
        u = M.widen(M.cast((C.spectrum(rng, r, c, kind) * 1e-3).astype(np.float32), "bf16"))
        want = M.orthogonalize(u)
        for dtype in dtypes:
            off = C.rms(M.orthogonalize_rounded(u, split=dtype == "f32") - want)
            with pytest.raises(AssertionError):
                C.check(rounded(u, dtype, **{lost: False}), want, off, dtype, kind)
