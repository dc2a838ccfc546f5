"""The unit's products as a training step uses them: experts' weights gathered,
forward, both gradients into the replicas, the shard step; the same unit
gathered in 8 bits; captured graphs, other streams, gradients against
differences."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import fsdp_oracle as O
from oracle import products_oracle as P
from tests.gpu_util import assert_bitexact, to_dev, to_host
from workloads.configs import ADAMW

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


def offsets_of(sizes):
    return torch.tensor(np.cumsum([0] + list(sizes)), dtype=torch.int32, device=DEV)


def randn(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def near(got, want, size, terms, what):
    """bf16 results of fp32 sums of `terms` products, in any order: 2^-8 of the
    value, and 2^-23 of the terms' magnitudes per addition."""
    err = (got.double() - want).abs()
    assert (err <= 2.0 ** -8 * want.abs() + 1.01 * terms * 2.0 ** -23 * size).all(), what


E, D, H = 4, 72, 136                         # experts, hidden, their inner size
SHAPES = [(D,), (E, H, D), (E, D, H)]        # a scale, W1 [out, in], W2
SIZES = [[30, 0, 51, 19], [1, 64, 0, 35], [100, 0, 0, 0]]


@pytest.mark.parametrize("layout", ["per_param", "flat"])
def test_a_step_of_experts(layout):
    """Three ranks, rows routed differently in each: forward and backward with
    the products, gradients in the replicas, then reduce-scatter and AdamW."""
    R, rows = 3, 100
    g = torch.Generator(device=DEV).manual_seed(1)
    plan, po = F.Plan(SHAPES, R, layout), O.plan_layout(SHAPES, R, layout)
    rng = np.random.default_rng(1)
    full = (rng.standard_normal(po.T) / 9).astype(np.float32)
    master_full = O.shard_pack(po, full)
    master = to_dev(master_full.reshape(-1))
    shards = torch.empty(R * plan.S, dtype=BF, device=DEV)
    F.fsdp_shard_pack(plan, to_dev(full), shards)
    recv = [torch.empty(plan.T, dtype=BF, device=DEV) for _ in range(R)]
    F.fsdp_gather_unflatten(plan, shards, recv)
    grads = [torch.full((plan.T,), float("nan"), dtype=BF, device=DEV) for _ in range(R)]
    for r in range(R):
        off = offsets_of(SIZES[r])
        _, w1, w2 = plan.unflatten(recv[r])
        ds, dw1, dw2 = plan.unflatten(grads[r])
        x, dy = randn(g, rows, D), randn(g, rows, D, scale=1e-2)
        h, y = (torch.empty(rows, n, dtype=BF, device=DEV) for n in (H, D))
        dh, dx = torch.empty_like(h), torch.empty_like(x)
        F.fsdp_grouped_matmul("nt", x, w1, h, off)
        a = torch.relu(h)
        F.fsdp_grouped_matmul("nt", a, w2, y, off)
        F.fsdp_grouped_matmul("nn", dy, w2, dh, off)
        F.fsdp_grouped_matmul("tn", dy, a, dw2, off)
        dh = dh * (h > 0)
        F.fsdp_grouped_matmul("nn", dh, w1, dx, off)
        F.fsdp_grouped_matmul("tn", dh, x, dw1, off)
        ds.copy_((dx * x).sum(0))
        lo = 0
        for e, n in enumerate(SIZES[r]):
            s = slice(lo, lo + n)
            lo += n
            # every product against 64 bits, on the operands that it had
            for got, p, q, terms in ((h[s], x[s], w1[e].T, D), (y[s], a[s], w2[e].T, H),
                                     (dx[s], dh[s], w1[e], H), (dw1[e], dh[s].T, x[s], n),
                                     (dw2[e], dy[s].T, a[s], n)):
                p, q = p.double(), q.double()
                near(got, p @ q, p.abs() @ q.abs(), terms, (r, e, got.shape))
        assert not torch.isnan(grads[r]).any()     # empty experts' gradients are zeros
    host = [to_host(t) for t in grads]
    m, v = torch.zeros_like(master), torch.zeros_like(master)
    F.fsdp_adamw_shard_step(plan, ADAMW, 1, grads, master, m, v, shards)
    zero = np.zeros_like(master_full)
    p2, m2, v2, param2 = O.shard_step(po, host, master_full, zero, zero, 1, ADAMW, "bf16")
    assert_bitexact(to_host(master).reshape(R, -1), p2, "master")
    assert_bitexact(to_host(shards).reshape(R, -1), param2, "param")


def test_a_unit_in_eight_bits():
    """The unit gathered as codes: forward and input gradient of every rank with
    them, against 64-bit products of the values that the codes stand for."""
    R, rows = 3, 100
    g = torch.Generator(device=DEV).manual_seed(2)
    plan = F.Plan(SHAPES, R, "per_param")
    shards = torch.empty(R * plan.S, dtype=BF, device=DEV)
    F.fsdp_shard_pack(plan, randn(g, plan.T, scale=0.1), shards)
    qu = F.Quant(plan)
    codes = [qu.code_buffer() for _ in range(R)]
    scales = [qu.scale_buffer() for _ in range(R)]
    rest = [qu.rest_buffer() for _ in range(R)]
    F.fsdp_gather_quantize(qu, shards, codes, scales, rest)
    units = [torch.empty(plan.T, dtype=torch.float32, device=DEV) for _ in range(R)]
    F.fsdp_dequantize(qu, codes, scales, rest, units)
    for r in range(R):
        off, sizes = offsets_of(SIZES[r]), SIZES[r]
        (c1, _), (s1, _) = qu.codes(codes[r]), qu.scales(scales[r])
        x, dy = randn(g, rows, D), randn(g, rows, H)
        xq = torch.empty(rows, 80, dtype=torch.int8, device=DEV)[:, :D]
        dq = torch.empty(rows, 144, dtype=torch.int8, device=DEV)[:, :H]
        sx, sd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        y, dx = torch.empty(rows, H, dtype=BF, device=DEV), torch.empty(rows, D, dtype=BF, device=DEV)
        F.fsdp_quantize_rows(x, xq, sx)
        F.fsdp_grouped_matmul_i8("nt", xq, sx, c1, s1, y, off)
        F.fsdp_quantize_rows(dy, dq, sd, channel=s1, offsets=off)
        F.fsdp_grouped_matmul_i8("nn", dq, sd, c1, None, dx, off)
        _, w1, _ = plan.unflatten(units[r])
        lo = 0
        for e, n in enumerate(sizes):
            s = slice(lo, lo + n)
            lo += n
            xc, xs = xq[s].double(), sx[s].double()[:, None]
            dc, ds = dq[s].double(), sd[s].double()[:, None]
            cw, sw = c1[e].double(), s1[e].double()[:, None]
            # the unit that was read back holds the rounded products
            assert ((w1[e].double() - cw * sw).abs() <= 2.0 ** -24 * (cw * sw).abs()).all()
            # (the codes' sums first: whole numbers, exact in 64 bits, zero
            # where they cancel)
            for got, want in ((y[s], (xc @ cw.T) * xs * sw.T), (dx[s], (dc @ cw) * ds)):
                # exact sums, three fp32 roundings (sum, two scales) and bf16's
                assert ((got.double() - want).abs() <=
                        (2.0 ** -8 + 4 * 2.0 ** -24) * want.abs()).all()
            # within half a step per entry of the unrounded layer
            full = x[s].double() @ (cw * sw).T
            most = sx[s].double()[:, None] / 2 * (cw * sw).abs().sum(1)
            # (half a step with the code's two fp32 roundings)
            assert ((y[s].double() - full).abs() <=
                    1.0001 * most + (2.0 ** -8 + 4 * 2.0 ** -24) * (full.abs() + most)).all()


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_gradients_are_differences(dtype):
    """f(W, x) = sum of v * (x W^T) is linear in each: with small integers f(W +
    dW) - f(W) = <grad W, dW> and the same for x, exactly."""
    g = torch.Generator(device=DEV).manual_seed(3)

    def ints(*s):
        return torch.randint(-2, 3, s, generator=g, device=DEV).to(dtype)
    sizes, n, k = [17, 0, 40], 24, 40
    off = offsets_of(sizes)
    W, dW, x, ddx, v = ints(3, n, k), ints(3, n, k), ints(57, k), ints(57, k), ints(57, n)

    def f(W, x):
        y = torch.empty(57, n, device=DEV)
        F.fsdp_grouped_matmul("nt", x, W, y, off)
        return (y.double() * v.double()).sum().item()
    gw, gx = torch.empty(3, n, k, device=DEV), torch.empty(57, k, device=DEV)
    F.fsdp_grouped_matmul("tn", v, x, gw, off)
    F.fsdp_grouped_matmul("nn", v, W, gx, off)
    assert f(W + dW, x) - f(W, x) == (gw.double() * dW.double()).sum().item()
    assert f(W, x + ddx) - f(W, x) == (gx.double() * ddx.double()).sum().item()


def calls(g):
    """Bound calls of every operator, their inputs (to be changed in place) and
    their outputs."""
    rows, n, k = 300, 136, 264
    sizes = [100, 0, 190, 10]
    off = offsets_of(sizes)
    x, w, dy = randn(g, rows, k), randn(g, 4, n, k), randn(g, rows, n)
    y, dx = torch.zeros(rows, n, dtype=BF, device=DEV), torch.zeros(rows, k, dtype=BF, device=DEV)
    dw, acc = torch.zeros(4, n, k, dtype=BF, device=DEV), torch.zeros(4, n, k, device=DEV)
    long_a, long_b = randn(g, 20000, 64), randn(g, 20000, 72)
    long_c = torch.zeros(64, 72, device=DEV)
    plan = F.Plan([(33, 40), (7,), (3, 5, 2100)], 3, "per_param")
    shards = randn(g, plan.R * plan.S)
    qu = F.Quant(plan)
    qu.prepare()
    codes = [qu.code_buffer().zero_() for _ in range(3)]
    scales = [qu.scale_buffer().zero_() for _ in range(3)]
    rest = [qu.rest_buffer().zero_() for _ in range(3)]
    units = [torch.zeros(plan.T, dtype=BF, device=DEV) for _ in range(3)]
    xq = torch.zeros(rows, 272, dtype=torch.int8, device=DEV)[:, :k]
    wq = torch.zeros(4, n, 272, dtype=torch.int8, device=DEV)[:, :, :k]
    sx, sw = torch.zeros(rows, device=DEV), torch.zeros(4 * n, device=DEV)
    yq = torch.zeros(rows, n, device=DEV)
    fs = [F.bind_grouped_matmul("nt", x, w, y, off), F.bind_grouped_matmul("nn", dy, w, dx, off),
          F.bind_grouped_matmul("tn", dy, x, dw, off),
          F.bind_grouped_matmul("tn", dy, x, acc, off, accumulate=True),
          F.bind_grouped_matmul("tn", long_a, long_b, long_c),
          F.bind_gather_quantize(qu, shards, codes, scales, rest),
          F.bind_dequantize(qu, codes, scales, rest, units),
          F.bind_quantize_rows(x, xq, sx),
          F.bind_quantize_rows(w.view(-1, k), wq.flatten(0, 1), sw),
          F.bind_grouped_matmul_i8("nt", xq, sx, wq, sw.view(4, n), yq, off)]
    return fs, [x, w, dy, long_a, long_b, shards], [y, dx, dw, acc, long_c, *codes, *scales, *rest,
                                                    *units, xq, sx, yq], acc


def test_captured_calls_replay():
    """A graph of all calls, replayed with changed inputs and eager work between
    the replays, against the eager calls."""
    g = torch.Generator(device=DEV).manual_seed(4)
    fs, inputs, outputs, acc = calls(g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        [f() for f in fs]
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        [f() for f in fs]
    for i in range(4):
        for t in inputs:
            t.copy_(randn(g, *t.shape))
        acc.zero_()
        [f() for f in fs]
        want = [t.clone() for t in outputs]
        for t in outputs:
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        junk = torch.randn(512, 512, device=DEV) @ torch.randn(512, 512, device=DEV)
        assert torch.isfinite(junk).all()
        for t, w in zip(outputs, want):
            assert torch.equal(t, w), i


def test_calls_on_another_stream():
    g = torch.Generator(device=DEV).manual_seed(5)
    fs, inputs, outputs, acc = calls(g)
    [f() for f in fs]
    torch.cuda.synchronize()
    want = [t.clone() for t in outputs]
    for t in outputs:
        t.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    [f(side) for f in fs]
    torch.cuda.current_stream().wait_stream(side)
    for t, w in zip(outputs, want):
        assert torch.equal(t, w)
    # the unbound form, whose workspace nobody else keeps
    a, b, c = inputs[3], inputs[4], torch.empty(64, 72, device=DEV)
    for s in (side, __import__("ctypes").c_void_p(side.cuda_stream)):
        c.zero_()
        side.wait_stream(torch.cuda.current_stream())
        F.fsdp_grouped_matmul("tn", a, b, c, stream=s)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(c, outputs[4])


def test_two_bindings_at_once():
    """Each has a workspace of its own."""
    g = torch.Generator(device=DEV).manual_seed(6)
    a, b = randn(g, 30000, 64), randn(g, 30000, 64)
    outs = [torch.zeros(64, 64, device=DEV) for _ in range(3)]
    fs = [F.bind_grouped_matmul("tn", a, b, outs[0]), F.bind_grouped_matmul("tn", b, a, outs[1]),
          F.bind_grouped_matmul("tn", a, a, outs[2])]
    [f() for f in fs]
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    streams = [torch.cuda.Stream() for _ in fs]
    for _ in range(5):
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        for f, s in zip(fs, streams):
            f(s)
        torch.cuda.synchronize()
        for t, w in zip(outs, want):
            assert torch.equal(t, w)


def test_results_do_not_change_from_call_to_call():
    g = torch.Generator(device=DEV).manual_seed(7)
    fs, _, outputs, acc = calls(g)
    [f() for f in fs]
    want = [t.clone() for t in outputs]
    for _ in range(3):
        acc.zero_()
        [f() for f in fs]
        assert all(torch.equal(t, w) for t, w in zip(outputs, want))


def test_a_gather_larger_than_the_caches():
    """Eight receivers of 42M codes each."""
    plan = F.Plan([(5130, 8192)], 8, "per_param")
    g = torch.Generator(device=DEV).manual_seed(8)
    full = randn(g, plan.T)
    shards = torch.empty(8 * plan.S, dtype=BF, device=DEV)
    F.fsdp_shard_pack(plan, full, shards)
    qu = F.Quant(plan)
    assert 8 * qu.code_bytes > 1 << 28
    codes, scales = [qu.code_buffer() for _ in range(8)], [qu.scale_buffer() for _ in range(8)]
    F.fsdp_gather_quantize(qu, shards, codes, scales, [qu.rest_buffer() for _ in range(8)])
    want, s = torch.empty(5130, 8192, dtype=torch.int8, device=DEV), torch.empty(5130, device=DEV)
    F.fsdp_quantize_rows(full.view(5130, 8192), want, s)
    for r in range(8):
        assert torch.equal(codes[r].view(5130, 8192), want) and torch.equal(scales[r], s)


def test_refusals_of_the_binding():
    x, w, y = (torch.zeros(*s, dtype=BF, device=DEV) for s in ((10, 16), (3, 24, 16), (10, 24)))
    off = offsets_of([4, 3, 3])
    mm = F.fsdp_grouped_matmul
    for args, match in [(("nt", x, w, y), "needs offsets"), (("nt", x, w, y, off[:3]), "elements"),
                        (("nt", x, w, y, off.long()), "int32"), (("nn", x, w, y, off), "fit"),
                        (("nt", x.float(), w, y, off), "one dtype"),
                        (("nt", x[:, ::2], w[..., :8], y, off), "contiguous"),
                        (("nt", x[0], w, y, off), "dimensions"),
                        (("nt", x.expand(10, 16)[:1].expand(10, 16), w, y, off), "overlap"),
                        (("tn", x, y, w, off), "fit"), (("nt", x, w, y[:9], off), "fit")]:
        with pytest.raises(ValueError, match=match):
            mm(*args)
    with pytest.raises(TypeError, match="dtype"):
        mm("nt", x.half(), w.half(), y, off)
    with pytest.raises(F.FsdpError):
        mm("nt", y[:, :16], w, y, off)     # the result on an operand
    with pytest.raises(ValueError, match="uint8"):
        mm("nt", x, w, y, off, workspace=torch.empty(9, device=DEV))
    q, s = torch.zeros(10, 16, dtype=torch.int8, device=DEV), torch.zeros(10, device=DEV)
    wq, sw = torch.zeros(24, 16, dtype=torch.int8, device=DEV), torch.zeros(24, device=DEV)
    m8 = F.fsdp_grouped_matmul_i8
    for args, match in [((x, s, wq, sw, y), "int8"), ((q, s[:9], wq, sw, y), "a_scale"),
                        ((q, s, wq, sw[:9], y), "b_scale"), ((q, s.double(), wq, sw, y), "a_scale"),
                        ((q[:, :12], s, wq[:, :12].contiguous(), sw, y), "multiple of 16"),
                        ((q, s, wq.expand(2, 24, 16), sw, y), "offsets|b_scale")]:
        with pytest.raises(ValueError, match=match):
            m8("nt", *args)
    qr = F.fsdp_quantize_rows
    for args, match in [((x, q[:9], s), "shape"), ((x, x, s), "int8"), ((x, q, s[:9]), "scales"),
                        ((x, torch.zeros(10, 24, dtype=torch.int8, device=DEV)[:, :16], s), "16"),
                        ((x, q, s, sw), "channel"), ((x, q, s, None, off.long()), "int32")]:
        with pytest.raises(ValueError, match=match):
            qr(*args)
