"""Groups without rows: what a weight gradient does with their results."""

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,k,rows,off", [(64, 64, 9000, 0), (70, 65, 9001, 1), (64, 64, 90, 0),
                                          (200, 300, 700, 0)])
def test_an_empty_groups_gradient_is_left(n, k, rows, off, out, dtype):
    """Added to, every bit of it stays (a -0 and a NaN's payload too), whether
    the sums are made in parts or not; not added to, it is +0."""
    g = torch.Generator(device=DEV).manual_seed(n)
    offsets = torch.tensor([0, 0, rows // 3, rows // 3, rows], dtype=torch.int32, device=DEV)
    a, b = (torch.randint(-3, 4, (rows * w + off,), generator=g, device=DEV).to(dtype)[off:]
            .view(rows, w) for w in (n, k))
    bits = torch.int16 if out == torch.bfloat16 else torch.int32
    c = torch.full((4, n, k), -0.0, dtype=out, device=DEV)
    odd = 0x7f81 if out == torch.bfloat16 else 0x7f800001   # a signalling NaN
    c.view(bits)[0, 0, ::3] = odd
    c.view(bits)[2, n - 1, ::2] = odd
    before = c.clone()
    F.fsdp_grouped_matmul("tn", a, b, c, offsets=offsets, accumulate=True)
    for e in (0, 2):
        assert torch.equal(c[e].view(bits), before[e].view(bits))
    for e, (lo, hi) in ((1, (0, rows // 3)), (3, (rows // 3, rows))):
        want = a[lo:hi].double().T @ b[lo:hi].double()
        assert torch.equal(c[e].double(), want.to(out).double())
    F.fsdp_grouped_matmul("tn", a, b, c, offsets=offsets)
    assert not c[0].view(bits).any() and not c[2].view(bits).any()
