"""How exact long fp32 sums are."""

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


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
@pytest.mark.parametrize("side,what", [(256, "32 x 32 tiles"), (1500, "64 x 64"),
                                       (2048, "128 x 128")])
@pytest.mark.parametrize("terms", [8192, 8161])
def test_long_sums_are_added_up_in_blocks(op, side, what, terms):
    """Normal numbers, 64 blocks of 128 terms.  With u = 2^-24, the most that one
    addition is off relative to its result, independent signs, and partial sums
    of i terms of variance i: a block is off by u^2 (1 + 2 + ... + 128), about u^2
    128^2 / 2, in the mean square, all 64 by u^2 8192 64, and their own sum by u^2
    128 (1 + 2 + ... + 64), about u^2 8192 32.  So the root of the mean square over
    the results' is at most u sqrt(96) = 5.8e-7; of 8192 terms in one go it would
    be u sqrt(8192 / 2) = 3.8e-6, and with roundings that are spread evenly over
    the step still 1 / sqrt(6) of that, 1.6e-6."""
    g = torch.Generator(device=DEV).manual_seed(terms + side)
    shapes = {"nt": ((side, terms), (side, terms)), "nn": ((side, terms), (terms, side)),
              "tn": ((terms, side), (terms, side))}[op]
    a, b = (torch.randn(s, generator=g, device=DEV) for s in shapes)
    c = torch.empty(side, side, device=DEV)
    F.fsdp_grouped_matmul(op, a, b, c)
    x = a.double().T if op == "tn" else a.double()
    want = x @ (b.double().T if op == "nt" else b.double())
    off = ((c.double() - want).square().mean() / want.square().mean()).sqrt().item()
    print(f"{op} {what}: {off:.2e}", flush=True)
    assert off < 2.0 ** -24 * 96 ** 0.5
