"""GPU parity of the unit's matrix products against 64-bit values: exact where
the numbers are small integers (every sum is then exact in fp32, in any order),
and within the roundings' bounds where they are not."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import products_oracle as P

pytestmark = pytest.mark.gpu
DEV = "cuda"
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu(request):
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    F.lib()
    print(f"[gpu] {request.node.name}", flush=True)
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


def offsets_of(sizes, first=0):
    return np.cumsum([first] + list(sizes)).astype(np.int32)


def matrix(x, dtype, off=0, pad=0):
    """A device matrix (or stack) with the values x, `off` elements into its
    allocation, rows `pad` elements further apart than they are long, and NaN in
    every place that is not its own."""
    x = np.asarray(x, np.float64)
    *lead, cols = x.shape
    n = int(np.prod(lead))
    buf = torch.full((off + n * (cols + pad) + 8,), float("nan"), dtype=TORCH[dtype], device=DEV)
    t = buf[off:off + n * (cols + pad)].view(*lead, cols + pad)[..., :cols]
    t.copy_(torch.from_numpy(x))
    return t


def shapes(op, rows, n, k, groups):
    return {"nt": ((rows, k), (groups, n, k), (rows, n)),
            "nn": ((rows, k), (groups, k, n), (rows, n)),
            "tn": ((rows, n), (rows, k), (groups, n, k))}[op]


def integers(rng, shape, most=4):
    return rng.integers(-most, most + 1, shape).astype(np.float64)


def exact_case(op, sizes, n, k, dtype="bf16", out="f32", off=0, pad=0, cpad=0, accumulate=False,
               first=0, tail=0, seed=0):
    """Integers: fp32 sums are exact below 2^24 (|terms| <= 16 here), so the
    result is, and a bf16 one is its rounding."""
    rng = np.random.default_rng(seed + n * 7 + k)
    rows = first + sum(sizes) + tail
    off_np = offsets_of(sizes, first)
    sa, sb, sc = shapes(op, rows, n, k, len(sizes))
    a, b, c = integers(rng, sa), integers(rng, sb), integers(rng, sc, 9)
    assert max(k, rows) * 16 < 2 ** 24
    want, _ = P.grouped(op, a, b, c, off_np, accumulate)
    # rows of no group may hold anything
    for x in ([a, b] if op == "tn" else [a]):
        x[:first] = np.nan
        x[first + sum(sizes):] = np.nan
    ta, tb, tc = matrix(a, dtype, off, pad), matrix(b, dtype, off, pad), matrix(c, out, 0, cpad)
    around = tc.untyped_storage()
    before = torch.tensor([], dtype=torch.uint8, device=DEV).set_(around).clone()
    offsets = torch.from_numpy(off_np).to(DEV)
    F.fsdp_grouped_matmul(op, ta, tb, tc, offsets=offsets, accumulate=accumulate)
    got = tc.double().cpu().numpy()
    w = torch.from_numpy(want).to(TORCH[out]).double().numpy()
    if not np.array_equal(got, w):
        bad = np.argwhere(got != w)
        raise AssertionError(f"{len(bad)} of {got.size} differ, first at {bad[0]}: "
                             f"{got[tuple(bad[0])]} not {w[tuple(bad[0])]}; last at {bad[-1]}")
    if cpad:     # nothing between the rows was written
        after = torch.tensor([], dtype=torch.uint8, device=DEV).set_(around).clone()
        tc.copy_(torch.from_numpy(np.asarray(c)))
        mine = torch.tensor([], dtype=torch.uint8, device=DEV).set_(around)
        assert torch.equal(mine, before)
        es = tc.element_size()
        keep = torch.ones(around.nbytes() // es, dtype=torch.bool, device=DEV)
        keep.as_strided(tc.shape, tc.stride(), tc.storage_offset()).fill_(False)
        keep = keep.repeat_interleave(es)
        assert torch.equal(after[keep], before[keep])


OPS = ["nt", "nn", "tn"]


@pytest.mark.parametrize("dtype,off,pad", [("bf16", 0, 0), ("bf16", 0, 8), ("bf16", 1, 0),
                                           ("bf16", 0, 3), ("f32", 0, 0), ("f32", 1, 3)])
@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("sizes,n,k", [
    ([1], 8, 8), ([1], 1, 1), ([5], 7, 3), ([64], 64, 64), ([65], 72, 136), ([130], 40, 200),
    ([3, 0, 17, 64, 1], 48, 72), ([0, 0, 33], 33, 65), ([2, 1, 0, 2], 129, 31),
    ([200, 1, 70], 136, 264)])
def test_small_products_are_exact(op, sizes, n, k, dtype, off, pad):
    exact_case(op, sizes, n, k, dtype=dtype, off=off, pad=pad)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype,n,k", [("bf16", 72, 136), ("bf16", 71, 133), ("f32", 71, 33)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_results_strides_and_rows_of_no_group(op, dtype, n, k, out, accumulate):
    """Rows before the first and behind the last group hold NaN and keep their
    results, and nothing between the rows of c is written."""
    exact_case(op, [40, 0, 90], n, k, dtype=dtype, out=out, cpad=5, first=3, tail=30,
               accumulate=accumulate)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("n,k,off", [(2056, 72, 0), (2051, 70, 0), (2056, 72, 1)])
def test_middle_tiles_are_exact(op, n, k, off):
    """Enough results for 128 x 128 tiles (tn: of n by 2,048)."""
    if op == "tn":
        exact_case(op, [70, 61], n, 2048 + k, off=off)
    else:
        exact_case(op, [700, 0, 1, 1400], n, k, off=off)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("off", [0, 1])
def test_fp32_in_larger_tiles(op, off):
    if op == "tn":
        exact_case(op, [70, 61], 2051, 2050, dtype="f32", off=off)
    else:
        exact_case(op, [700, 0, 1, 1400], 2051, 70, dtype="f32", off=off)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("k", [72, 200])
def test_large_tiles_are_exact(op, k):
    """Enough results for 256 x 256 tiles."""
    if op == "tn":
        exact_case(op, [k, 9, 0], 2056, 2824)
    else:
        exact_case(op, [2600, 3, 0, 1900], 4104, k)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n", [([2100, 0, 1990], 4104), ([1700, 300, 2500, 1], 3900),
                                     ([4096], 4352), ([129, 4095], 4352)])
def test_the_last_tiles_cut(op, sizes, n):
    """A few 256 x 256 tiles more than fill the card: cut in two or four; groups
    that end in the first or the second half of a tile."""
    exact_case(op, sizes, n, 136)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k", [([16], 40, 600), ([7, 0, 30, 1, 2], 200, 1096),
                                       ([1], 4104, 4096), ([3] * 70, 72, 264)])
def test_few_rows(op, sizes, n, k):
    """16 rows per group or fewer, and one group with more."""
    exact_case(op, sizes, n, k)
    exact_case(op, sizes, n, k, out="bf16", accumulate=True, cpad=3, first=1, tail=2)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k", [([777], 1000, 2056), ([70, 0, 200, 1, 300], 328, 4100),
                                       ([640], 72, 2048)])
def test_long_sums_of_few_tiles(op, sizes, n, k):
    """More rows than the thin tiles take, fewer 64 x 64 tiles than compute
    units, sums of 4 KiB and more: the waves of a tile share the sum."""
    exact_case(op, sizes, n, k)
    exact_case(op, sizes, n, k, out="bf16", accumulate=True, cpad=3, first=1, tail=2)


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_many_groups(op):
    """More groups than a wave has lanes, most of them empty."""
    rng = np.random.default_rng(3)
    sizes = [int(rng.integers(0, 40)) if rng.random() < 0.3 else 0 for _ in range(200)]
    exact_case(op, sizes, 24, 40)


def test_weight_gradients_of_many_groups():
    rng = np.random.default_rng(4)
    sizes = [int(rng.integers(0, 90)) if rng.random() < 0.5 else 0 for _ in range(150)]
    exact_case("tn", sizes, 24, 40)


@pytest.mark.parametrize("n,k,rows,off", [(64, 64, 9000, 0), (200, 72, 20000, 0),
                                          (70, 65, 9001, 1)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_weight_gradients_in_parts(n, k, rows, off, accumulate):
    """Long sums of few results: made in parts and joined."""
    sizes = [rows // 3, 0, rows - rows // 3]
    a = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    assert F.grouped_matmul_workspace("tn", a, torch.empty(rows, k, dtype=torch.bfloat16,
                                                           device=DEV),
                                      torch.empty(3, n, k, device=DEV)) is not None
    exact_case("tn", sizes, n, k, off=off, accumulate=accumulate)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_roundings(op, dtype, out):
    """Any numbers.  A sum of k terms in fp32, in any order and with additions
    off by up to a step each, is off by at most k 2^-23 of the terms' magnitudes;
    the result's rounding by half a step of it (2^-8 in bf16, 2^-24 in fp32)."""
    rng = np.random.default_rng(11)
    sizes = [70, 0, 131]
    n, k, rows = 136, 264, 201
    sa, sb, sc = shapes(op, rows, n, k, 3)
    vals = [torch.from_numpy(rng.standard_normal(s)).to(TORCH[dtype]) for s in (sa, sb)]
    off = offsets_of(sizes)
    want, size = P.grouped(op, *(v.double().numpy() for v in vals), np.zeros(sc), off)
    c = torch.empty(sc, dtype=TORCH[out], device=DEV)
    F.fsdp_grouped_matmul(op, vals[0].to(DEV), vals[1].to(DEV), c,
                          offsets=torch.from_numpy(off).to(DEV))
    terms = max(sizes) if op == "tn" else k
    half = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[out]
    err = np.abs(c.double().cpu().numpy() - want)
    assert (err <= half * np.abs(want) + (1 + half) * terms * 2.0 ** -23 * size).all()


@pytest.mark.parametrize("op", ["nt", "nn"])
def test_one_weight_needs_no_offsets(op):
    rng = np.random.default_rng(2)
    a, b = integers(rng, (50, 40)), integers(rng, (24, 40) if op == "nt" else (40, 24))
    c = torch.full((50, 24), 7.0, device=DEV)
    F.fsdp_grouped_matmul(op, matrix(a, "bf16"), matrix(b, "bf16"), c)
    assert np.array_equal(c.cpu().numpy(), a @ (b.T if op == "nt" else b))


def test_nothing_to_do():
    e = torch.empty
    c = e(0, 8, device=DEV)
    F.fsdp_grouped_matmul("nt", e(0, 16, device=DEV), e(8, 16, device=DEV), c)
    w = torch.full((2, 8, 16), 5.0, device=DEV)
    offsets = torch.zeros(3, dtype=torch.int32, device=DEV)
    for dt in (torch.float32, torch.bfloat16):
        a, b = e(0, 8, dtype=dt, device=DEV), e(0, 16, dtype=dt, device=DEV)
        F.fsdp_grouped_matmul("tn", a, b, w, offsets=offsets, accumulate=True)
        assert (w == 5.0).all()
        F.fsdp_grouped_matmul("tn", a, b, w, offsets=offsets)
        assert (w == 0.0).all()
        w.fill_(5.0)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_infinities_stay_in_their_rows(op, dtype):
    """An infinity in one row of a reaches that row's results (of tn: that
    column's) and no others; as the sum's end is filled up with zeros, the rows
    and groups beside it stay finite."""
    rng = np.random.default_rng(8)
    sizes, n, k = [30, 41], 40, 72
    sa, sb, sc = shapes(op, 71, n, k, 2)
    a, b = np.abs(integers(rng, sa)) + 1, np.abs(integers(rng, sb)) + 1
    a[29, 5] = np.inf
    c = torch.zeros(sc, device=DEV)
    F.fsdp_grouped_matmul(op, matrix(a, dtype), matrix(b, dtype), c,
                          offsets=torch.from_numpy(offsets_of(sizes)).to(DEV))
    bad = ~torch.isfinite(c)
    want = torch.zeros_like(bad)
    if op == "tn":
        want[0, 5] = True
    else:
        want[29] = True
    assert torch.equal(bad, want)


# -------------------------------------------------------------- 8-bit codes
def codes_matrix(x):
    """Codes with rows padded to 16 bytes by zeros."""
    *lead, cols = x.shape
    t = torch.zeros(*lead, -(-cols // 16) * 16, dtype=torch.int8, device=DEV)[..., :cols]
    t.copy_(torch.from_numpy(x))
    return t


def i8_case(op, sizes, n, k, out="f32", accumulate=False, first=0, tail=0, scales=True, garbage=False):
    rng = np.random.default_rng(n + k)
    rows, E = first + sum(sizes) + tail, len(sizes)
    sa_, sb_, sc = shapes(op, rows, n, k, E)
    a, b = (rng.integers(-127, 128, s).astype(np.int8) for s in (sa_, sb_))
    sa = np.exp(rng.standard_normal(rows)).astype(np.float32)
    sb = np.exp(rng.standard_normal((E, n))).astype(np.float32) if scales else None
    c = torch.from_numpy(rng.standard_normal(sc)).to(TORCH[out])
    off = offsets_of(sizes, first)
    want = P.grouped_i8(op, a, sa, b, sb, c.float().numpy(), off, accumulate)
    c = c.to(DEV)
    tb = codes_matrix(b)
    if garbage:     # behind b's rows: only a's padding has to be zero
        whole = tb.as_strided((*tb.shape[:-1], tb.stride(-2)), tb.stride())
        whole[..., tb.shape[-1]:] = 77
    F.fsdp_grouped_matmul_i8(op, codes_matrix(a), torch.from_numpy(sa).to(DEV), tb,
                             None if sb is None else torch.from_numpy(sb).to(DEV), c,
                             offsets=torch.from_numpy(off).to(DEV), accumulate=accumulate)
    got, w = c.float().cpu().numpy(), torch.from_numpy(want).to(TORCH[out]).float().numpy()
    if not np.array_equal(got, w):
        bad = np.argwhere(got != w)
        raise AssertionError(f"{len(bad)} of {got.size} differ, first at {bad[0]}: "
                             f"{got[tuple(bad[0])]} not {w[tuple(bad[0])]}; last at {bad[-1]}")


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k", [
    ([1], 16, 16), ([1], 1, 1), ([5], 7, 3), ([64], 64, 128), ([65], 72, 136), ([130], 40, 1000),
    ([3, 0, 17, 64, 1], 48, 72), ([0, 0, 33], 33, 65), ([2, 1, 0, 2], 129, 31),
    ([200, 1, 70], 136, 264)])
def test_products_of_codes_are_exact(op, sizes, n, k):
    i8_case(op, sizes, n, k, garbage=True)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("scales", [False, True])
def test_products_of_codes_results(op, out, accumulate, scales):
    i8_case(op, [40, 0, 90], 71, 133, out=out, accumulate=accumulate, first=3, tail=30,
            scales=scales)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("n,k", [(2056, 72), (2051, 70), (4104, 200)])
def test_products_of_codes_in_larger_tiles(op, n, k):
    i8_case(op, [700, 0, 1, 1400] if n < 4000 else [2600, 3, 0, 1900], n, k)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k", [([2100, 0, 1990], 4104, 136), ([129, 4095], 4352, 200),
                                       ([7, 0, 30, 1, 2], 200, 1096), ([1], 4104, 4099),
                                       ([3] * 70, 71, 263)])
def test_products_of_codes_last_tiles_and_few_rows(op, sizes, n, k):
    i8_case(op, sizes, n, k)
    if sum(sizes) < 300:
        i8_case(op, sizes, n, k, out="bf16", accumulate=True, first=1, tail=2, scales=False)


@pytest.mark.parametrize("op", ["nt", "nn"])
@pytest.mark.parametrize("sizes,n,k", [([777], 1000, 4112), ([70, 0, 200, 1, 300], 329, 5001),
                                       ([640], 72, 4096)])
def test_products_of_codes_long_sums_of_few_tiles(op, sizes, n, k):
    i8_case(op, sizes, n, k)
    i8_case(op, sizes, n, k, out="bf16", accumulate=True, first=1, tail=2, scales=False)


def test_codes_longest_sum():
    """The largest sum there can be, 131,072 times 127 squared, is exact."""
    k = 131072
    a = torch.full((3, k), 127, dtype=torch.int8, device=DEV)
    b = torch.full((5, k), -127, dtype=torch.int8, device=DEV)
    one = torch.ones(3, device=DEV)
    c = torch.empty(3, 5, device=DEV)
    F.fsdp_grouped_matmul_i8("nt", a, one, b, None, c)
    assert (c == float(np.float32(-127 * 127 * k))).all()


def test_a_row_without_a_scale_is_nan():
    a = torch.ones(4, 16, dtype=torch.int8, device=DEV)
    sa = torch.tensor([1.0, float("nan"), 0.0, 2.0], device=DEV)
    c = torch.empty(4, 3, dtype=torch.bfloat16, device=DEV)
    F.fsdp_grouped_matmul_i8("nt", a, sa, torch.ones(3, 16, dtype=torch.int8, device=DEV),
                             torch.tensor([1.0, 2.0, 3.0], device=DEV), c)
    want = torch.tensor([[16., 32., 48.], [float("nan")] * 3, [0.] * 3, [32., 64., 96.]])
    assert torch.equal(torch.nan_to_num(c.float().cpu(), 9e9), torch.nan_to_num(want, 9e9))
