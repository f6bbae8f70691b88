"""The 8-bit product's kernel for one row, which takes the scales apart itself
and quantizes a row of bf16 for itself: NaN bytes, bytes at both ends, rows with
infinities and NaN, and the largest and smallest values."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_fp8 import BF16, E4M3, E5M2, F32, _pair, _random, _values

pytestmark = pytest.mark.gpu

# (n, k): one group and many, pieces of 1024 that end inside, ragged last groups
SIZES = [(1, 1), (2, 128), (41, 300), (300, 1025), (301, 2049), (64, 4096), (33, 5000)]


def _bits(t):
    return t.view(torch.int16 if t.dtype == BF16 else torch.int32)


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_nan_scales(n, k, kind):
    """A NaN byte in the row makes every output NaN, one in a row of b its own."""
    require_gpu()
    groups = (k + 127) // 128
    for at in sorted({0, groups // 2, groups - 1}):
        a, b = _pair(1, n, k, n + k, kind)
        want = (_values(a) @ _values(b).t()).float()
        assert torch.equal(F.flashopt_byte_product(a, b, F32), want)
        for row in sorted({0, n // 2, n - 1}):
            keep = b.scales[row, at].clone()
            b.scales[row, at] = 255
            bad = torch.arange(n, device="cuda")[None] == row
            for dtype in (F32, BF16):
                got = F.flashopt_byte_product(a, b, dtype)
                assert torch.equal(torch.isnan(got), bad) and torch.equal(got[~bad], want.to(dtype)[~bad])
            b.scales[row, at] = keep
        a.scales[0, at] = 255
        assert torch.isnan(F.flashopt_byte_product(a, b, F32)).all()
        a.codes.view(torch.uint8)[:] = 0                       # NaN times codes of zero, too
        assert torch.isnan(F.flashopt_byte_product(a, b)).all()


@pytest.mark.parametrize("n,k", SIZES)
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_scales_at_both_ends(n, k, kind):
    """The sum of the two exponents is what counts: products of integers of at
    most 8 under 2^-127, multiples of it, are fp32 values."""
    require_gpu()
    groups = (k + 127) // 128
    a, b = _pair(1, n, k, n + k, kind)
    for sa, sb in ((0, 254), (254, 0), (0, 127), (127, 0), (254, 1), (1, 254), (64, 190)):
        a.scales[:, :groups], b.scales[:, :groups] = sa, sb
        assert torch.equal(F.flashopt_byte_product(a, b, F32).double(), _values(a) @ _values(b).t())
    a.scales[:, :groups], b.scales[:, :groups] = 0, 0          # 2^-254 of small integers: below fp32's range
    assert (F.flashopt_byte_product(a, b, F32) == 0).all()
    # 2^127 and 2^200 times integers: from 2^128 on an infinity.  (One product:
    # sums in fp32 may meet infinities of both signs where the whole is finite.)
    for sb in (127, 200) if k == 1 else ():
        a.scales[:, :groups], b.scales[:, :groups] = 254, sb
        assert torch.equal(F.flashopt_byte_product(a, b, F32), (_values(a) @ _values(b).t()).float())


@pytest.mark.parametrize("k", [1, 8, 130, 1000, 1024, 2500, 4096, 14336])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_are_not_finite(k, dtype):
    """An infinity or NaN anywhere in the row: every output NaN, and the bits of
    the quantization and the product one by one."""
    require_gpu()
    w = F.flashopt_byte_quantize(_random(77, k, 5, BF16, 2), block=True)
    for bad in (float("inf"), float("-inf"), float("nan")):
        for at in sorted({0, min(k - 1, 130), k // 2, k - 1}):
            x = _random(1, k, 4, dtype, 2)
            x[0, at] = bad
            for out in (BF16, F32):
                y = F.flashopt_byte_linear(x, w, out)
                assert torch.isnan(y).all()
                assert torch.equal(_bits(y), _bits(F.flashopt_byte_product(F.flashopt_byte_quantize(x), w, out)))


@pytest.mark.parametrize("k", [1, 8, 130, 1000, 1024, 2500, 4096])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_at_the_ends_of_the_range(k, dtype):
    """The largest and smallest values, zeros of both signs, and groups of each
    beside one another: as quantized and multiplied one by one, bit for bit."""
    require_gpu()
    w = F.flashopt_byte_quantize(_random(77, k, 5, BF16, 2), block=True)
    top, low = torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal
    x = _random(1, k, 4, dtype, 2)
    sizes = torch.tensor([1.0, top / 2 ** 12, low, low / 64, 0.0, 1e-20, 1e20], dtype=torch.float64, device="cuda")
    mixed = x.double() * sizes[(torch.arange(k, device="cuda") // 128) % 7]
    rows = [mixed, torch.full_like(mixed, top), torch.full_like(mixed, -top), mixed * 0.0, -(mixed * 0.0).abs(),
            torch.full_like(mixed, low / 64)]
    for row in rows:
        x = row.to(dtype)
        assert torch.isfinite(x).all()
        q = F.flashopt_byte_quantize(x)
        for out in (BF16, F32):
            got, want = F.flashopt_byte_linear(x, w, out), F.flashopt_byte_product(q, w, out)
            assert torch.equal(_bits(got), _bits(want))
