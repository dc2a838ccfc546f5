"""The 8-bit gather's kernels that small units do not reach: codes that pass the
caches by, for few and for many receivers, of both types, in rows longer than a
workgroup holds."""

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


@pytest.mark.parametrize("layout", ["per_param", "flat"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,rows,cols", [(5, 411, 131072), (13, 160, 131072), (13, 5130, 4099),
                                         (8, 60001, 563)])
def test_gathers_larger_than_the_caches(R, rows, cols, dtype, layout):
    plan = F.Plan([(rows, cols), (7,)], R, layout)
    g = torch.Generator(device=DEV).manual_seed(R)
    full = torch.randn(plan.T, generator=g, device=DEV).to(dtype)
    shards = torch.empty(R * plan.S, dtype=dtype, device=DEV)
    F.fsdp_shard_pack(plan, full, shards)
    qu = F.Quant(plan)
    assert R * qu.code_bytes > 1 << 28
    codes = [torch.full((qu.code_bytes,), 99, dtype=torch.int8, device=DEV) for _ in range(R)]
    scales = [qu.scale_buffer() for _ in range(R)]
    rest = [qu.rest_buffer(dtype) for _ in range(R)]
    F.fsdp_gather_quantize(qu, shards, codes, scales, rest)
    x = full[:rows * cols].view(rows, cols)
    want = torch.full((qu.code_bytes,), 99, dtype=torch.int8, device=DEV)
    s = torch.empty(rows, device=DEV)
    F.fsdp_quantize_rows(x, qu.codes(want)[0], s)
    for r in range(R):
        assert torch.equal(codes[r], want) and torch.equal(scales[r], s)
        assert torch.equal(rest[r], full[-7:])
    unit = torch.empty(plan.T, device=DEV)
    F.fsdp_dequantize(qu, codes, scales, rest, [unit] + [None] * (R - 1))
    assert torch.equal(unit[:rows * cols].view(rows, cols),
                       qu.codes(want)[0].float() * s[:, None])
    assert torch.equal(unit[-7:], full[-7:].float())
