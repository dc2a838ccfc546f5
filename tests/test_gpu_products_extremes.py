"""Calls of the products and of the 8-bit codes at the ends of what they take: the
most groups and receivers, rows and matrices further apart than 32 bits count, and
offsets that change between the replays of a graph."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def integers(seed, *shape, dtype=BF, most=4):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-most, most + 1, shape, generator=g, device=DEV).to(dtype)


def plain(op, a, b, c, offsets):
    """The product in 64 bits, exact for small integers, as c's type."""
    out = c.double()
    a, b = a.double(), b.double()
    for g, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        if op == "tn":
            out[g] = a[lo:hi].T @ b[lo:hi]
        elif hi > lo:
            out[lo:hi] = a[lo:hi] @ (b[g].T if op == "nt" else b[g])
    return out.to(c.dtype)


def operands(op, rows, n, k, groups, dtype=BF):
    sa, sb, sc = {"nt": ((rows, k), (groups, n, k), (rows, n)),
                  "nn": ((rows, k), (groups, k, n), (rows, n)),
                  "tn": ((rows, n), (rows, k), (groups, n, k))}[op]
    return integers(1, *sa, dtype=dtype), integers(2, *sb, dtype=dtype), torch.zeros(sc, device=DEV)


# ------------------------------------------------------------ the most groups
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
def test_65536_groups(op, dtype):
    """Of which 300 have rows, the first and the last among them."""
    rng = np.random.default_rng(5)
    E = 65536
    sizes = np.zeros(E, np.int64)
    have = np.concatenate([[0, E - 1], rng.choice(np.arange(1, E - 1), 298, replace=False)])
    sizes[have] = rng.integers(1, 40, 300)
    offsets = np.cumsum(np.concatenate([[0], sizes])).astype(np.int32)
    a, b, c = operands(op, int(offsets[-1]), 24, 16, E, dtype)
    F.fsdp_grouped_matmul(op, a, b, c, torch.from_numpy(offsets).to(DEV))
    for g in have:
        lo, hi = offsets[g], offsets[g + 1]
        if op == "tn":
            assert torch.equal(c[g], (a[lo:hi].double().T @ b[lo:hi].double()).float()), g
        else:
            w = b[g].double().T if op == "nt" else b[g].double()
            assert torch.equal(c[lo:hi], (a[lo:hi].double() @ w).float()), g
    if op == "tn":
        c[torch.from_numpy(have).to(DEV)] = 0
        assert not c.any()


def test_65536_groups_of_codes():
    E, rows, k = 65536, 500, 32
    sizes = torch.zeros(E, dtype=torch.int64)
    sizes[[0, 7, 64, 40000, E - 1]] = torch.tensor([100, 1, 99, 250, 50])
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]).int()
    group = torch.repeat_interleave(torch.arange(E), sizes).to(DEV)
    x, channel = integers(3, rows, k), integers(4, E, k, dtype=torch.float32).abs_() + 1
    codes, s = torch.zeros(rows, k, dtype=torch.int8, device=DEV), torch.zeros(rows, device=DEV)
    F.fsdp_quantize_rows(x, codes, s, channel=channel, offsets=offsets.to(DEV))
    want, sw = torch.zeros_like(codes), torch.zeros_like(s)
    F.fsdp_quantize_rows(x.float() * channel[group], want, sw)
    assert torch.equal(codes, want) and torch.equal(s, sw)
    w = integers(5, 1, 16, k, dtype=torch.int8, most=127).expand(E, 16, k)   # one for all
    c = torch.zeros(rows, 16, device=DEV)
    F.fsdp_grouped_matmul_i8("nt", codes, s, w, None, c, offsets.to(DEV))
    assert torch.equal(c, (codes.double() @ w[0].double().T).float() * s[:, None])


# ----------------------------------------------------- beyond 32 bits of elements
FAR = (1 << 22) - 8     # elements: rows of bf16 just below 8 MiB apart


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
@pytest.mark.parametrize("cols", [(72, 136), (71, 133)])
def test_rows_far_apart(op, cols):
    """1,100 rows 8 MiB apart: 4.6e9 elements from the first to the last."""
    rows, (n, k) = 1100, cols
    assert rows * FAR > 2 ** 32
    off = [0, 513, 513, rows]
    a, b, c = operands(op, rows, n, k, 3)
    block = torch.empty(rows * FAR, dtype=BF, device=DEV)
    far_a = block.as_strided((rows, a.shape[1]), (FAR, 1), 0)
    far_a.copy_(a)
    if op == "tn":
        far_b = block.as_strided((rows, k), (FAR, 1), 1024)
        far_b.copy_(b)
        far_c = c
    else:
        far_b = b
        out = torch.empty(rows * FAR, dtype=BF, device=DEV)
        far_c = out.as_strided((rows, n), (FAR, 1), 16)
    F.fsdp_grouped_matmul(op, far_a, far_b, far_c,
                          torch.tensor(off, dtype=torch.int32, device=DEV))
    assert torch.equal(far_c, plain(op, a, b, far_c, off))


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
def test_matrices_far_apart(op):
    """Three groups' matrices 2.2e9 elements apart."""
    n, k, off, stride = 200, 136, [0, 70, 71, 300], 2_200_000_008
    a, b, c = operands(op, 300, n, k, 3)
    stacked = c if op == "tn" else b
    block = torch.empty(2 * stride + stacked[0].numel(), dtype=BF, device=DEV)
    far = block.as_strided(stacked.shape, (stride, stacked.shape[2], 1))
    far.copy_(stacked)
    args = (a, b, far) if op == "tn" else (a, far, c)
    F.fsdp_grouped_matmul(op, *args, torch.tensor(off, dtype=torch.int32, device=DEV))
    assert torch.equal(args[2], plain(op, a, b, args[2], off))


def test_rows_of_codes_far_apart():
    """x, its codes, and the product's operand and result."""
    rows, k, n, far = 700, 100, 72, (1 << 23) - 16
    assert rows * far > 2 ** 32
    x = integers(6, rows, k)
    x[:, 0] = 127.0
    block = torch.empty(rows * far, dtype=torch.int8, device=DEV)
    codes = block.as_strided((rows, k), (far, 1))
    wide = torch.empty(rows * far // 2, dtype=BF, device=DEV)
    xs = wide.as_strided((rows, k), (far // 2, 1), 3)
    xs.copy_(x)
    s = torch.empty(rows, device=DEV)
    F.fsdp_quantize_rows(xs, codes, s)
    assert torch.equal(codes.float(), x.float()) and torch.equal(s, torch.full_like(s, 127.0) / 127)
    w = torch.zeros(n, 112, dtype=torch.int8, device=DEV)[:, :k]
    w.copy_(integers(7, n, k, dtype=torch.int8, most=127))
    c = wide.as_strided((rows, n), (far // 2, 1), 1024)
    F.fsdp_grouped_matmul_i8("nt", codes, s, w, None, c)
    assert torch.equal(c, (x.double() @ w.double().T).to(BF))


# --------------------------------------------------------- graphs and their offsets
def test_replays_with_other_offsets():
    """The groups' sizes are read when the call runs: a graph captured with some
    serves all others, among them none at all and everything in one group."""
    rows, n, k, E = 9000, 72, 64, 3
    a, b = integers(8, rows, k), integers(9, E, n, k)
    dy = integers(10, rows, n)
    y, dw = torch.zeros(rows, n, device=DEV), torch.zeros(E, n, k, device=DEV)
    acc = torch.zeros(E, n, k, device=DEV)
    q, s = torch.zeros(rows, k, dtype=torch.int8, device=DEV), torch.zeros(rows, device=DEV)
    channel = integers(11, E, k, dtype=torch.float32).abs_() + 1
    offsets = torch.tensor([0, 100, 5000, rows], dtype=torch.int32, device=DEV)
    fs = [F.bind_grouped_matmul("nt", a, b, y, offsets),
          F.bind_grouped_matmul("tn", dy, a, dw, offsets),
          F.bind_grouped_matmul("tn", dy, a, acc, offsets, accumulate=True),
          F.bind_quantize_rows(a, q, s, channel, offsets)]
    outputs = (y, dw, acc, q, s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        [f() for f in fs]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        [f() for f in fs]
    for off in ([0, 100, 5000, rows], [0, 0, 0, 0], [0, rows, rows, rows], [17, 17, 17, 18],
                [0, 3000, 3000, 8999], [0, 1, 2, 3]):
        offsets.copy_(torch.tensor(off, dtype=torch.int32))
        for t in outputs:
            t.fill_(1)
        [f() for f in fs]
        want = [t.clone() for t in outputs]
        assert torch.equal(y, plain("nt", a, b, torch.ones_like(y), off))
        assert torch.equal(dw, plain("tn", dy, a, dw, off))
        assert torch.equal(acc, dw + 1)
        for t in outputs:
            t.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        assert all(torch.equal(t, w) for t, w in zip(outputs, want)), off


# ---------------------------------------------------------------- the most receivers
@pytest.mark.parametrize("layout", ["per_param", "flat"])
def test_64_receivers(layout):
    R = 64
    plan = F.Plan([(100, 33), (5,), (3, 2500)], R, layout)
    full = torch.randn(plan.T, device=DEV)
    shards = torch.empty(R * plan.S, device=DEV)
    F.fsdp_shard_pack(plan, full, shards)
    qu = F.Quant(plan)
    codes, scales = ([make() for _ in range(R)] for make in (qu.code_buffer, qu.scale_buffer))
    rest = [qu.rest_buffer(torch.float32) for _ in range(R)]
    F.fsdp_gather_quantize(qu, shards, codes, scales, rest)
    for r in range(1, R):
        assert torch.equal(codes[r], codes[0]) and torch.equal(scales[r], scales[0])
        assert torch.equal(rest[r], full[3300:3305])
    units = [torch.empty(plan.T, dtype=BF, device=DEV) for _ in range(R)]
    F.fsdp_dequantize(qu, codes, scales, rest, units)
    w = codes[0][:100 * 48].view(100, 48)[:, :33].float() * scales[0][:100, None]
    assert torch.equal(units[63][:3300].view(100, 33), w.to(BF))
    # receivers may share what they read
    again = [torch.empty(plan.T, dtype=BF, device=DEV) for _ in range(R)]
    F.fsdp_dequantize(qu, codes[:1] * R, scales[:1] * R, rest[:1] * R, again)
    assert all(torch.equal(u, units[0]) for u in units + again)
