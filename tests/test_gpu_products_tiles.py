"""Every kernel of the unit's products, by products that are known to get it:
exact, as their numbers are small integers."""

import pytest
import torch

import fully_sharded_amd as F
from tests.products_tiles import CASES
from tests.test_gpu_products import exact_case, i8_case

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("name", CASES)
def test_each_kernel_is_exact(name):
    op, kind, sizes, n, k, off = CASES[name]
    if kind == "i8":
        i8_case(op, sizes, n, k, garbage=True)
        i8_case(op, sizes, n, k, out="bf16", accumulate=True)
    else:
        exact_case(op, sizes, n, k, dtype=kind, off=off)
        exact_case(op, sizes, n, k, dtype=kind, off=off, out="bf16", accumulate=True)
