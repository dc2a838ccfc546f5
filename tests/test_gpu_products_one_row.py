"""Products with an operand of one long row, 8 MiB and more: exact, as the numbers
are small integers."""

import pytest
import torch

import fully_sharded_amd as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
LONG = 1 << 22
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def integers(seed, *shape, off=0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    n = 1
    for s in shape:
        n *= s
    return torch.randint(-4, 5, (n + off,), generator=g, device=DEV).to(dtype)[off:].view(shape)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,k,off", [(LONG, 8, 0), (8, LONG, 0), (LONG + 1, 3, 1), (3, LONG + 5, 0)])
def test_one_tokens_gradient(n, k, off, dtype):
    a, b = (integers(s, 1, w, off=off, dtype=DTYPE[dtype]) for s, w in ((1, n), (2, k)))
    c = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    F.fsdp_grouped_matmul("tn", a, b, c)
    assert torch.equal(c.float(), a.float().T * b.float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,off", [(LONG, 0), (LONG + 3, 1)])
def test_a_sum_of_one_term(n, off, dtype):
    """Weights of one row each, by group."""
    a = integers(3, 7, 1, dtype=DTYPE[dtype])
    b = integers(4, 2, 1, n, off=off, dtype=DTYPE[dtype])
    c = torch.full((7, n), 9.0, device=DEV)
    F.fsdp_grouped_matmul("nn", a, b, c, torch.tensor([1, 3, 6], dtype=torch.int32, device=DEV))
    assert (c[0] == 9.0).all() and (c[6] == 9.0).all()
    assert torch.equal(c[1:3], a[1:3].float() * b[0].float())
    assert torch.equal(c[3:6], a[3:6].float() * b[1].float())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("k,off", [(LONG, 0), (LONG + 7, 1)])
def test_one_dot_product(k, off, dtype):
    """A sum of 4.2 million terms of 0 or 1, exact in fp32."""
    a, b = (integers(s, 1, k, off=off, dtype=DTYPE[dtype]).clamp_(0, 1) for s in (5, 6))
    c = torch.empty(1, 1, device=DEV)
    F.fsdp_grouped_matmul("nt", a, b, c)
    assert c.item() == (a.double() * b.double()).sum().item()


def test_one_row_of_codes():
    n = 1 << 23
    a, b = (integers(s, r, w).to(torch.int8) for s, r, w in ((7, 3, 16), (8, 1, n)))
    a[:, 1:] = 0
    sa, c = torch.tensor([1.0, 2.0, 0.5], device=DEV), torch.empty(3, n, device=DEV)
    F.fsdp_grouped_matmul_i8("nn", a[:, :1], sa, b, None, c)
    assert torch.equal(c, a[:, :1].float() * b.float() * sa[:, None])
