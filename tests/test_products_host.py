"""Host-side checks of the unit's products and 8-bit codes (no GPU): sizes and
places, and every entry point's refusals, which come before any device call."""

import ctypes

import pytest
import torch

import fully_sharded_amd as F
from fully_sharded_amd import binding as B

BASE = 1 << 40   # addresses that are never touched: every call here is refused
FAR = 1 << 36


def at(i, off=0):
    return ctypes.c_void_p(BASE + i * FAR + off)


def shape(kind="nt", /, groups=2, rows=10, n=24, k=40, **more):
    cols = {"nt": (k, k, n), "nn": (k, n, n), "tn": (n, k, k)}[kind]
    m = B.MatmulShape({"nt": 0, "nn": 1, "tn": 2}[kind], groups, rows, n, k, *cols, n * k, 0, 0)
    for name, v in more.items():
        setattr(m, name, v)
    return m


def matmul(m, offsets=at(0), a=at(1), b=at(2), dtype=1, c=at(3), out=1, ws=None, n=0):
    return B.lib().fsdp_grouped_matmul(None if m is None else ctypes.byref(m), offsets, a, b, dtype,
                                       c, out, ws, n, None)


@pytest.mark.parametrize("op", ["nt", "nn", "tn"])
def test_matmul_refusals(op):
    bad = [dict(op=3), dict(op=-1), dict(groups=0), dict(rows=-1), dict(n=0), dict(k=0),
           dict(lda=7), dict(ldb=7), dict(ldc=7), dict(group_stride=-1), dict(accumulate=2)]
    if op == "tn":
        bad.append(dict(group_stride=24 * 40 - 1))
    for more in bad:
        assert matmul(shape(op, **more)) == -1, more
    big = 1 << 30
    side = 1 << 26
    for more in [dict(groups=65537), dict(rows=big), dict(n=big, lda=big, ldb=big, ldc=big,
                                                          group_stride=big * 40),
                 dict(n=side, lda=side, ldb=side, ldc=side, group_stride=side * 40),
                 dict(k=side, lda=side, ldb=side, ldc=side, group_stride=side * 24),
                 # lengths that no array has, and 64 bits do not hold
                 dict(lda=1 << 55), dict(ldb=1 << 55), dict(lda=1 << 62), dict(ldb=1 << 62),
                 dict(ldc=1 << 62, group_stride=(1 << 63) - 1),
                 dict(group_stride=(1 << 63) - 1, groups=60000)]:
        assert matmul(shape(op, **more)) == -2, more
    m = shape(op)
    assert matmul(None) == -1
    for more in [dict(a=None), dict(b=None), dict(c=None), dict(dtype=2), dict(out=-1),
                 dict(offsets=None), dict(a=at(1, 1)), dict(b=at(2, 1)), dict(c=at(3, 1)),
                 dict(c=at(3, 2), out=0), dict(a=at(1, 2), dtype=0), dict(offsets=at(0, 2)),
                 dict(c=at(1)), dict(c=at(2, 16)), dict(c=at(0)),     # c on what is read
                 dict(c=at(0, 8)), dict(a=at(3, 16))]:
        assert matmul(m, **more) == -1, more


def test_matmul_grids():
    """More tiles than a launch takes are refused, before anything is read."""
    assert matmul(shape("nt", groups=1, rows=1 << 29, n=1 << 26, k=8, group_stride=0)) == -2
    assert matmul(shape("tn", groups=60000, rows=8, n=1 << 14, k=1 << 14)) == -2


def test_workspace():
    L, n = B.lib(), ctypes.c_int64(-7)

    def need(m, dtype=1):
        assert L.fsdp_grouped_matmul_workspace(ctypes.byref(m), dtype, ctypes.byref(n)) == 0
        return n.value
    assert need(shape("nt")) == need(shape("nn")) == need(shape("tn")) == 0
    long = shape("tn", groups=1, rows=100000, n=64, k=64)
    size = need(long)
    assert size > 0 and size % 256 == 0 and need(long, 0) == 0
    for more in [dict(ws=None, n=size), dict(ws=at(4), n=size - 1), dict(ws=at(4, 128), n=size),
                 dict(ws=at(1), n=size), dict(ws=at(3), n=size), dict(ws=at(0), n=size)]:
        assert matmul(long, **more) == -1, more
    assert L.fsdp_grouped_matmul_workspace(None, 1, ctypes.byref(n)) == -1
    assert L.fsdp_grouped_matmul_workspace(ctypes.byref(long), 2, ctypes.byref(n)) == -1
    assert L.fsdp_grouped_matmul_workspace(ctypes.byref(long), 1, None) == -1
    assert L.fsdp_grouped_matmul_workspace(ctypes.byref(shape("nt", k=0)), 1,
                                           ctypes.byref(n)) == -1


def i8(m, offsets=at(0), a=at(1), sa=at(4), b=at(2), sb=at(5), stride=24, c=at(3), out=1):
    return B.lib().fsdp_grouped_matmul_i8(ctypes.byref(m), offsets, a, sa, b, sb, stride, c, out,
                                          None)


def codes_shape(kind, /, **more):
    m = shape(kind, lda=48, ldb=48 if kind == "nt" else 32, group_stride=48 * 40)
    for name, v in more.items():
        setattr(m, name, v)
    return m


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_codes_refusals(op):
    for more in [dict(op=2), dict(lda=40), dict(ldb=41), dict(lda=56), dict(group_stride=8),
                 dict(groups=0), dict(k=0), dict(accumulate=-1)]:
        assert i8(codes_shape(op, **more)) == -1, more
    wide = 1 << 23
    for more in [dict(k=131073, lda=1 << 18, ldb=1 << 18), dict(lda=wide), dict(ldb=wide)]:
        assert i8(codes_shape(op, **more)) == -2, more
    m = codes_shape(op)
    for more in [dict(a=None), dict(sa=None), dict(b=None), dict(c=None), dict(offsets=None),
                 dict(out=5), dict(a=at(1, 8)), dict(b=at(2, 8)), dict(sa=at(4, 2)),
                 dict(sb=at(5, 1)), dict(c=at(3, 1)), dict(stride=-1), dict(c=at(1)),
                 dict(c=at(2)), dict(c=at(4)), dict(c=at(5)), dict(c=at(0))]:
        assert i8(m, **more) == -1, more


def rows(x=at(1), dtype=1, n=10, cols=40, ldx=40, channel=at(2), stride=40, offsets=at(3),
         groups=2, codes=at(4), ldc=48, scales=at(5)):
    return B.lib().fsdp_quantize_rows(x, dtype, n, cols, ldx, channel, stride, offsets, groups,
                                      codes, ldc, scales, None)


def test_quantize_rows_refusals():
    for more in [dict(dtype=2), dict(n=-1), dict(cols=0), dict(ldx=39), dict(groups=0),
                 dict(stride=-1), dict(ldc=47), dict(ldc=32), dict(offsets=None), dict(x=None),
                 dict(codes=None), dict(scales=None), dict(x=at(1, 1)), dict(codes=at(4, 8)),
                 dict(scales=at(5, 2)), dict(channel=at(2, 2)), dict(offsets=at(3, 1)),
                 dict(codes=at(1)), dict(scales=at(1)), dict(scales=at(4)), dict(codes=at(2)),
                 dict(codes=at(3)), dict(scales=at(3))]:
        assert rows(**more) == -1, more
    for more in [dict(n=1 << 24), dict(cols=(1 << 30) + 1, ldx=1 << 31, ldc=1 << 31),
                 dict(groups=65537), dict(ldx=1 << 60), dict(ldc=1 << 60), dict(stride=1 << 60)]:
        assert rows(**more) == -2, more
    assert rows(n=0) == 0 and rows(n=0, x=None, codes=None, scales=None) == 0


SHAPES = [(6, 4), (5,), (3, 2, 7), (9, 1), (1, 33)]


def handle(plan, params):
    h = ctypes.c_void_p()
    arr = (ctypes.c_int32 * max(1, len(params)))(*params)
    return B.lib().fsdp_quant_plan(plan.handle, len(params), arr, ctypes.byref(h)), h


def test_choice_of_parameters():
    plan = F.Plan(SHAPES, 3, "per_param")
    assert F.Quant(plan).params == [0, 2, 3, 4]
    assert F.fsdp_quant_plan(plan, [3, 0]).params == [3, 0]
    for bad in ([], [1], [0, 0], [5], [-1], [0, 1]):
        st, h = handle(plan, bad)
        assert st == -1 and not h.value, bad
    assert B.lib().fsdp_quant_plan(None, 1, (ctypes.c_int32 * 1)(0),
                                   ctypes.byref(ctypes.c_void_p())) == -1
    assert B.lib().fsdp_quant_plan(plan.handle, 1, None, ctypes.byref(ctypes.c_void_p())) == -1
    assert B.lib().fsdp_quant_plan(plan.handle, 1, (ctypes.c_int32 * 1)(0), None) == -1
    st, h = handle(F.Plan([(1, (1 << 30) + 1), (2, 2)], 1, "flat"), [0])
    assert st == -2 and not h.value
    B.lib().fsdp_quant_destroy(None)


@pytest.mark.parametrize("layout", ["per_param", "flat"])
def test_places_and_views(layout):
    plan = F.Plan(SHAPES, 3, layout)
    qu = F.Quant(plan, [4, 0, 2])
    assert (qu.code_bytes, qu.n_scales, qu.rest_numel) == (6 * 16 + 6 * 16 + 48, 6 + 6 + 1, 14)
    codes = torch.arange(qu.code_bytes, dtype=torch.int32).to(torch.int8)
    a, b, c = qu.codes(codes)
    assert (a.shape, b.shape, c.shape) == ((1, 33), (6, 4), (3, 2, 7))
    assert b.stride() == (16, 1) and c.stride() == (32, 16, 1)
    assert a.data_ptr() == codes.data_ptr() + 192 and c[2, 1, 6] == codes[96 + 5 * 16 + 6]
    scales = torch.arange(13.0)
    s = qu.scales(scales)
    assert [tuple(x.shape) for x in s] == [(1,), (6,), (3, 2)]
    assert s[0].tolist() == [12.0] and s[2][2, 1] == 11.0
    r = qu.rest(torch.arange(14.0))
    assert [tuple(x.shape) for x in r] == [(5,), (9, 1)] and r[1][0, 0] == 5.0


def test_quant_queries_refuse():
    L, out = B.lib(), (ctypes.c_int64 * 5)()
    qu = F.Quant(F.Plan(SHAPES, 2, "flat"))
    assert L.fsdp_quant_sizes(None, out) == -1 and L.fsdp_quant_sizes(qu.handle, None) == -1
    assert L.fsdp_quant_param(None, 0, out) == -1 and L.fsdp_quant_param(qu.handle, 0, None) == -1
    assert L.fsdp_quant_param(qu.handle, 5, out) == -1
    assert L.fsdp_quant_param(qu.handle, -1, out) == -1
    assert L.fsdp_quant_prepare(None, None) == -1


def ptrs(*v):
    return (ctypes.c_void_p * len(v))(*[None if x is None else x.value for x in v])


def test_gather_quantize_refusals():
    qu = F.Quant(F.Plan(SHAPES, 2, "flat"))
    codes, scales, rest = ptrs(at(1), at(2)), ptrs(at(3), at(4)), ptrs(at(5), at(6))

    def call(shards=at(0), dtype=1, codes=codes, scales=scales, rest=rest, h=qu.handle):
        return B.lib().fsdp_gather_quantize(h, shards, dtype, codes, scales, rest, None)
    for more in [dict(h=None), dict(shards=None), dict(dtype=2), dict(codes=None),
                 dict(scales=None), dict(rest=None), dict(shards=at(0, 1)),
                 dict(scales=ptrs(at(3), None)), dict(rest=ptrs(None, at(6))),
                 dict(codes=ptrs(at(1), at(2, 8))), dict(scales=ptrs(at(3, 2), at(4))),
                 dict(rest=ptrs(at(5, 1), at(6))), dict(codes=ptrs(at(1), at(1))),
                 dict(scales=ptrs(at(3), at(1))), dict(rest=ptrs(at(5), at(3))),
                 dict(codes=ptrs(at(0), at(2)))]:
        assert call(**more) == -1, more
    assert call(codes=ptrs(None, None)) == 0      # nobody receives


def test_dequantize_refusals():
    qu = F.Quant(F.Plan(SHAPES, 2, "flat"))
    codes, scales, rest = ptrs(at(1), at(2)), ptrs(at(3), at(4)), ptrs(at(5), at(6))
    full = ptrs(at(7), at(8))

    def call(codes=codes, scales=scales, rest=rest, rdt=1, full=full, dt=1, h=qu.handle):
        return B.lib().fsdp_dequantize(h, codes, scales, rest, rdt, full, dt, None)
    for more in [dict(h=None), dict(codes=None), dict(scales=None), dict(rest=None),
                 dict(full=None), dict(rdt=2), dict(dt=-1), dict(codes=ptrs(None, at(2))),
                 dict(scales=ptrs(at(3), None)), dict(rest=ptrs(None, at(6))),
                 dict(full=ptrs(at(7, 1), at(8))), dict(full=ptrs(at(7), at(7))),
                 dict(full=ptrs(at(1), at(8))), dict(full=ptrs(at(7), at(3))),
                 dict(full=ptrs(at(6), at(8)))]:
        assert call(**more) == -1, more
    assert call(full=ptrs(None, None), codes=ptrs(None, None)) == 0


def test_the_binding_refuses_host_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        F.fsdp_grouped_matmul("nt", x, x, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="op is one of"):
        F.fsdp_grouped_matmul("tt", x, x, x)
    with pytest.raises(ValueError, match="op is one of"):
        F.fsdp_grouped_matmul_i8("tn", x, x, x, x, x)
    with pytest.raises(ValueError, match="GPU"):
        F.fsdp_quantize_rows(x, x, x)
    qu = F.Quant(F.Plan(SHAPES, 2, "flat"))
    with pytest.raises(ValueError, match="R\\*S"):
        F.fsdp_gather_quantize(qu, x, [None] * 2, [None] * 2, [None] * 2)
    with pytest.raises(ValueError, match="R buffers"):
        F.fsdp_gather_quantize(qu, torch.zeros(2 * qu.plan.S), [None], [None] * 2, [None] * 2)
    with pytest.raises(ValueError, match="need a unit"):
        F.fsdp_dequantize(qu, [None] * 2, [None] * 2, [None] * 2, [None] * 2)
