"""8-bit codes of the largest and smallest numbers that have any."""

import numpy as np
import pytest
import torch

import fully_sharded_amd as F
from oracle import products_oracle as P
from tests.gpu_util import to_dev

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


def quantized(bits):
    r, c = bits.shape
    codes = torch.zeros(r, -(-c // 16) * 16, dtype=torch.int8, device=DEV)
    scales = torch.empty(r, device=DEV)
    F.fsdp_quantize_rows(to_dev(bits), codes[:, :c], scales)
    return codes[:, :c].cpu().numpy(), scales.cpu().numpy()


@pytest.mark.parametrize("top", [127, 126, 125, 0, -99, -100])
def test_bf16_codes_are_the_exact_roundings_at_every_size(top):
    """Every pair of 8-bit significands, the largest entry between 2^top and twice
    that, the others 14 binades below at most.  A quotient x 127 / a is a tie or at
    least 2^-(9 + j) from one, j the binades between.  Three roundings of 2^-24 move
    it by less than 2^(7 - j) 2^-22; above 2^126, where 1 / a is below fp32's normal
    numbers (spaced by 2^-149, and above 2^-128), its rounding is 2^-22 and all three
    are less than 2^(7 - j) 2^-21 = 2^-(14 + j).  So but for ties the codes are the
    exact roundings."""
    sig = np.arange(128, 256)
    a = np.repeat(sig[:, None] << 14, 128 * 15, 1)
    x = np.broadcast_to((sig[:, None] << np.arange(15)[None, :]).reshape(1, -1), a.shape)
    x = np.concatenate([sig[:, None] << 14, np.where(x > a, 0, x)], 1).astype(np.int64)
    den = 2 * x[:, :1]
    low, rest = x * 254 // den, x * 254 % den
    want = low + ((2 * rest > den) | ((2 * rest == den) & (low % 2 == 1)))
    values = np.ldexp(x.astype(np.float64), top - 21).astype(np.float32)
    bits = P.cast(values, "bf16")
    assert np.array_equal(P.widen(bits), values) and np.isfinite(values).all()
    got, scales = quantized(bits)
    tie = 2 * rest == den
    assert np.array_equal(got[~tie], want[~tie])
    assert ((got[tie] == low[tie]) | (got[tie] == low[tie] + 1)).all()
    # a (1 / 127): two roundings of half a step
    exact = values[:, 0].astype(np.float64) / 127
    assert (np.abs(scales - exact) <= exact * 2.0 ** -24 * 2.001).all()


@pytest.mark.parametrize("top", [127, 126, -100])
def test_fp32_codes_at_every_size(top):
    """Bit for bit as documented, and within 127 2^-21 of half a step of x 127 / a."""
    rng = np.random.default_rng(abs(top))
    x = np.ldexp(rng.uniform(-1, 1, (40, 3000)), top).astype(np.float32)
    x[:, 0] = np.ldexp(rng.uniform(1, 1.99, 40), top).astype(np.float32)
    x[0, 0] = np.float32(2.0 ** top)
    codes, scales = P.quantize(x)
    got, s = quantized(x)
    assert np.array_equal(got, codes) and np.array_equal(s.view(np.uint32), scales.view(np.uint32))
    quotient = x.astype(np.float64) * 127 / np.abs(x).max(1, keepdims=True)
    assert (np.abs(got - quotient) <= 0.5 + 127 * 2.0 ** -21).all()
