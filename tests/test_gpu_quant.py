"""GPU parity of the 8-bit codes: rows quantised, a unit gathered in 8 bits and
read back, bit for bit with the oracle."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import fsdp_oracle as O
from oracle import products_oracle as P
from tests.gpu_util import to_dev, to_host

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


def values(rng, shape, dtype, sigma=1.0):
    return P.cast((rng.standard_normal(shape) * sigma).astype(np.float32), dtype)


def quantized(x, dtype, off=0, pad=0, channel=None, offsets=None, rows=None):
    """fsdp_quantize_rows of the oracle's values; codes and scales start at 99."""
    r, c = x.shape
    buf = to_dev(np.zeros(off + r * (c + pad) + 8, x.dtype))
    t = buf[off:off + r * (c + pad)].view(r, c + pad)[:, :c]
    t.copy_(to_dev(x))
    whole = torch.full((r, -(-c // 16) * 16 + 16), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((r,), 99.0, device=DEV)
    F.fsdp_quantize_rows(t, whole[:, :c], scales,
                         None if channel is None else to_dev(channel),
                         None if offsets is None else to_dev(offsets))
    return whole.cpu().numpy(), scales.cpu().numpy()


def check_codes(whole, scales, codes, want, c, rows=slice(None)):
    padded = -(-c // 16) * 16
    assert np.array_equal(whole[rows, :c], codes[rows])
    assert (whole[rows, c:padded] == 0).all() and (whole[:, padded:] == 99).all()
    assert np.array_equal(scales[rows].view(np.uint32), want[rows].view(np.uint32))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off,pad", [(0, 0), (1, 0), (0, 3)])
@pytest.mark.parametrize("r,c", [(1, 1), (3, 7), (5, 16), (9, 333), (6, 512), (3, 2048),
                                 (4, 2049), (2, 4096), (3, 14336), (2, 16384), (2, 16391),
                                 (1, 40000)])
def test_rows(r, c, off, pad, dtype):
    rng = np.random.default_rng(r * c)
    x = values(rng, (r, c), dtype)
    codes, scales = P.quantize(P.widen(x))
    check_codes(*quantized(x, dtype, off, pad), codes, scales, c)


@pytest.mark.parametrize("c", [40, 5000, 17000])
def test_rows_that_have_no_scale(c):
    """Zeros, tiny rows, infinities and NaN; the largest and smallest values."""
    rng = np.random.default_rng(c)
    x = rng.standard_normal((9, c)).astype(np.float32)
    x[1] = 0
    x[2] *= 2.0 ** -120
    x[3, c // 2] = np.inf
    x[4, c - 1] = np.nan
    x[5] *= 1e-45 / np.abs(x[5]).max()
    x[6, 3] = np.finfo(np.float32).max
    x[7] = np.float32(2.0 ** -100)
    x[8, 0] = -np.inf
    codes, scales = P.quantize(x)
    whole, got = quantized(x, "f32")
    assert np.array_equal(np.isnan(got), np.isnan(scales))
    check_codes(whole, np.where(np.isnan(got), np.float32(0), got),
                codes, np.where(np.isnan(scales), np.float32(0), scales), c)


def test_bf16_codes_are_the_exact_roundings():
    """Every pair of 8-bit significands, 14 binades apart at most, against the
    exact quotient 127 x / a.  With x = xs 2^e, a = as 2^f and j = f - e >= 0 the
    quotient times 2 as 2^j is a whole number, and so is a tie's (2 c + 1) / 2, so
    it is a tie or at least 1 / (2 as 2^j) >= 2^-(9 + j) from one.  The code is
    the rounding of x fl(fl(1 / a) 127) in fp32: three roundings of 2^-24 each move
    it by less than 2^(7 - j) 2^-22 = 2^-(15 + j).  So it is the exact rounding, but
    for ties, where the product may be on either side and both neighbours are
    half a step off."""
    sig = np.arange(128, 256).astype(np.float64)
    a = sig[:, None, None] * 2.0 ** 14
    x = (sig[None, :, None] * 2.0 ** np.arange(0, 15)[None, None, :])
    x = np.broadcast_to(np.where(x > a, 0, x), (128, 128, 15)).reshape(128, -1)
    x = np.concatenate([sig[:, None] * 2.0 ** 14, x], 1)
    num, den = (x * 254).astype(np.int64), (2 * sig[:, None] * 2.0 ** 14).astype(np.int64)
    low = num // den
    twice = 2 * (num - low * den)
    want = low + ((twice > den) | ((twice == den) & (low % 2 == 1)))
    bits = P.cast(x.astype(np.float32), "bf16")
    assert np.array_equal(P.widen(bits).astype(np.float64), x)
    whole, _ = quantized(bits, "bf16")
    got, tie = whole[:, :x.shape[1]], twice == den
    assert np.array_equal(got[~tie], want[~tie])
    assert tie.any() and ((got[tie] == low[tie]) | (got[tie] == low[tie] + 1)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("c", [24, 333, 3000])
def test_rows_by_channel_and_group(c, dtype):
    rng = np.random.default_rng(c)
    off = np.array([2, 2, 5, 5, 11, 14], np.int32)
    r = 17
    x = values(rng, (r, c), dtype)
    channel = np.exp(rng.standard_normal((5, c))).astype(np.float32)
    group = np.searchsorted(off, np.arange(r), side="right") - 1
    mine = (np.arange(r) >= 2) & (np.arange(r) < 14)
    codes, scales = P.quantize(P.widen(x), channel[np.clip(group, 0, 4)])
    whole, got = quantized(x, dtype, channel=channel, offsets=off)
    check_codes(whole, got, codes, scales, c, rows=mine)
    assert (whole[~mine] == 99).all() and (got[~mine] == 99).all()
    # one channel vector for all rows
    codes, scales = P.quantize(P.widen(x), channel[0])
    check_codes(*quantized(x, dtype, channel=channel[0]), codes, scales, c)


UNIT = [(33, 7), (5,), (3, 2, 40), (9, 1), (1, 2500), (130, 66), (2,), (17, 129), (4, 512)]


@pytest.mark.parametrize("layout", ["per_param", "flat"])
@pytest.mark.parametrize("R", [1, 2, 3, 8, 13])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("params", [None, [7, 2]])
def test_gather_and_read_back(R, layout, dtype, params):
    rng = np.random.default_rng(R)
    po, plan = O.plan_layout(UNIT, R, layout), F.Plan(UNIT, R, layout)
    full = values(rng, po.T, dtype)
    shards = to_dev(O.shard_pack(po, full).reshape(-1))
    qu = F.Quant(plan, params)
    chosen = qu.params
    codes = [torch.full((qu.code_bytes,), 99, dtype=torch.int8, device=DEV) for _ in range(R)]
    scales = [qu.scale_buffer() for _ in range(R)]
    rest = [qu.rest_buffer(TORCH[dtype]) for _ in range(R)]
    skipped = R // 2 if R > 2 else None
    take = [None if r == skipped else codes[r] for r in range(R)]
    F.fsdp_gather_quantize(qu, shards, take, scales, rest)
    at = np.cumsum([0] + [int(np.prod(s)) for s in UNIT])
    want = {"bf16": P.widen(full).copy(), "f32": P.widen(full).copy()}
    for r in range(R):
        if r == skipped:
            assert (codes[r] == 99).all()
            continue
        for view, sc, p in zip(qu.codes(codes[r]), qu.scales(scales[r]), chosen):
            x = P.widen(full[at[p]:at[p + 1]]).reshape(-1, UNIT[p][-1])
            c, s = P.quantize(x)
            assert view.shape == UNIT[p] and view.stride(-2) % 16 == 0
            assert np.array_equal(view.cpu().numpy().reshape(c.shape), c)
            assert np.array_equal(sc.cpu().numpy().reshape(-1).view(np.uint32), s.view(np.uint32))
            whole = codes[r].as_strided((len(s), view.stride(-2)), (view.stride(-2), 1),
                                        view.storage_offset())
            assert (whole[:, UNIT[p][-1]:] == 0).all()
            want["f32"][at[p]:at[p + 1]] = (c.astype(np.float32) * s[:, None]).reshape(-1)
        others = [p for p in range(len(UNIT)) if p not in chosen]
        for view, p in zip(qu.rest(rest[r]), others):
            assert np.array_equal(to_host(view).reshape(-1), full[at[p]:at[p + 1]])
    if skipped is not None:      # read back from another receiver's buffers
        for b in (codes, scales, rest):
            b[skipped] = b[0]
    for out in ("bf16", "f32"):
        units = [torch.full((po.T,), 99.0, dtype=TORCH[out], device=DEV) for _ in range(R)]
        leave = None if R == 1 else R - 1
        F.fsdp_dequantize(qu, codes, scales, rest,
                          [None if r == leave else u for r, u in enumerate(units)])
        w = P.cast(want["f32"], out)
        for r, u in enumerate(units):
            if r == leave:
                assert (u == 99).all()
            else:
                assert np.array_equal(to_host(u), w)
