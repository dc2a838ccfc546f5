"""Sums of 8-bit codes at the ends of their range."""

import pytest
import torch

import fully_sharded_amd as F

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("rows,n", [(3, 5), (70, 200), (300, 136)])
@pytest.mark.parametrize("x,y,k", [(-128, -128, 131071), (-128, 127, 131072), (127, 127, 131072),
                                   (-127, 127, 131072)])
def test_the_longest_sums(op, rows, n, x, y, k):
    """131,071 squares of -128 are 2^31 - 2^14, a number of fp32; 131,072 of 127, and
    of -128 times 127, are less than 2^31 and rounded once."""
    a = torch.zeros(rows, 131072, dtype=torch.int8, device=DEV)[:, :k]
    shape = (n, 131072) if op == "nt" else (k, -(-n // 16) * 16)
    b = torch.zeros(shape, dtype=torch.int8, device=DEV)[:, :k if op == "nt" else n]
    a.fill_(x)
    b.fill_(y)
    c = torch.empty(rows, n, device=DEV)
    F.fsdp_grouped_matmul_i8(op, a, torch.ones(rows, device=DEV), b, None, c)
    assert (c == torch.tensor(float(x * y * k), dtype=torch.float32, device=DEV)).all()
