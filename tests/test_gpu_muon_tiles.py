"""Every tile that the products of an orthogonalisation take (32, 64, 128 and
256 on a side, in A, B, X' and the last step, for bf16 results and for fp32
ones) against 64-bit values, at sides that leave tiles part full."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import muon_oracle as M
from tests import muon_check as C
from tests.muon_units import UNITS
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


def exact(u):
    """The definition in 64 bits, products of two matrices each."""
    a, b, c = M.POLY
    x = torch.from_numpy(u).to("cuda").double()
    x = x / (torch.linalg.norm(x) + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.T.contiguous() if tall else x
    for _ in range(5):
        g = x @ x.T.contiguous()
        x = a * x + (b * g + c * (g @ g)) @ x
    return (x.T if tall else x).cpu().numpy()


@pytest.mark.parametrize("udt,odt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("name", UNITS)
def test_units_of_each_tile(name, udt, odt):
    """All matrices of the unit; what the precision costs is imitated on the
    first of each shape, the others have the same distribution."""
    shapes = list(UNITS[name][0]) + [(33,)]
    rng = np.random.default_rng(len(shapes))
    us = [rng.standard_normal(s, dtype=np.float32) * 1e-3 for s in shapes]
    offs = {}
    for k, (u, got) in enumerate(run_ortho(shapes, us, udt, odt)):
        want = exact(u)
        if u.shape not in offs:
            offs[u.shape] = C.rms(M.orthogonalize_rounded(u, split=odt == "f32") - want)
        C.check(got, want, offs[u.shape], odt, f"matrix {k}")
