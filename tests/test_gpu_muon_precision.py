"""The precision of bf16 results of the orthogonalisation, held to that of their
rounding: diagonals or low parts that were lost would show."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import muon_oracle as M
from tests import muon_check as C
from tests.test_gpu_muon import run_ortho

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("udt", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["white", "low", "steep"])
@pytest.mark.parametrize("r,c", [(63, 64), (64, 64), (65, 64), (65, 191), (100, 333), (333, 100),
                                 (128, 128), (129, 129), (257, 255), (40, 1025), (1025, 40),
                                 (320, 960), (700, 512)])
def test_bf16_results_are_near_their_rounding(r, c, kind, udt):
    rng = np.random.default_rng(r * 1000 + c)
    (u, got), = run_ortho([(r, c)], [C.spectrum(rng, r, c, kind) * 1e-3], udt, "bf16")
    want = M.orthogonalize(u)
    C.check(got, want, C.rms(M.orthogonalize_rounded(u) - want), "bf16", f"{kind} {udt}")
