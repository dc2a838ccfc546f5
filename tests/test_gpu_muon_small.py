"""The orthogonalisation of updates whose norm is far below eps, and steps that
shrink their matrix: the operands keep their bits there too."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import muon_oracle as M
from tests.test_gpu_muon import check, run_ortho, spectrum

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()


@pytest.mark.parametrize("udt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("r,c", [(1, 1), (3, 40), (96, 160), (257, 255), (700, 600)])
def test_norm_below_eps(r, c, udt, odt):
    """|U| from eps down to 1e-24 of it, one matrix a call."""
    rng = np.random.default_rng(r + c)
    for k, ratio in enumerate((1.0, 1e-2, 1e-4, 1e-6, 1e-8, 1e-9, 1e-14, 1e-24)):
        u = spectrum(rng, r, c, ("white", "low")[k % 2])
        u *= 1e-7 * ratio / np.linalg.norm(u)
        (v, got), = run_ortho([(r, c)], [u], udt, odt)
        check(got, v, odt, what=f"|U| = {ratio} eps")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_matrices_of_every_size_in_one_unit(dt):
    """Each matrix has exponents of its own: small, ordinary and zero ones
    beside each other."""
    rng = np.random.default_rng(31)
    shapes = [(512, 512), (100, 333), (333, 100), (512, 512), (64, 64), (9, 5)]
    size = (1e-3, 1e-16, 1e-12, 1e-20, 0.0, 1e-9)
    us = [rng.standard_normal(s) * z for s, z in zip(shapes, size)]
    for off in (0, 1):
        for k, (u, got) in enumerate(run_ortho(shapes, us, dt, dt, off=off)):
            if size[k] == 0:
                assert (M.widen(got) == 0).all()
            else:
                check(got, u, dt, what=f"matrix {k}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_steps_that_shrink(dt):
    rng = np.random.default_rng(32)
    u = rng.standard_normal((96, 160)) * 1e-3
    for steps, poly in ((16, (0.25, 0.0, 0.0)), (7, (0.1, -0.05, 0.01)), (3, (0.0, 1.0, 0.0)),
                        (4, (0.02, 0.0, 1.0))):
        hp = dict(F.MUON, steps=steps, coefficients=poly)
        (v, got), = run_ortho([(96, 160)], [u], dt, dt, hp)
        check(got, v, dt, steps, poly=poly, what=f"{steps} steps of {poly}")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_results_below_the_types_range_are_zero(dt):
    """eps far above any update, and powers that leave no singular value."""
    rng = np.random.default_rng(33)
    u = rng.standard_normal((70, 90))
    for hp in (dict(F.MUON, eps=1e300), dict(F.MUON, eps=1e60),
               dict(F.MUON, steps=8, coefficients=(0.0, 1.0, 0.0)),
               dict(F.MUON, steps=16, coefficients=(0.0, 0.0, 1e-3))):
        (_, got), = run_ortho([(70, 90)], [u], dt, dt, hp)
        assert (M.widen(got) == 0).all()
