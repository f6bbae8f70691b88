"""The MXFP4 product and linear layer at the borders between their kernels."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("n,k", [(4096, 8192), (4096, 8200), (4097, 4096), (4097, 4104), (8192, 4096), (8192, 4104),
                                 (8193, 7168), (8193, 7176), (16384, 7168), (16384, 7176), (16385, 3584),
                                 (16385, 3592)])
def test_few_rows_on_both_sides_of_the_linear_rule(n, k):
    """Quantized in the product and before it: the same values, one K step
    more or less, one workgroup more or less to a CU."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(n + k)
    w = F.flashopt_mx_quantize(torch.randn(n, k, generator=g, device="cuda"))
    for m in (1, 4, 5):
        x = torch.randn(m, k, generator=g, device="cuda").to(BF16)
        apart = torch.empty(m, k + 1, dtype=BF16, device="cuda")[:, 1:].copy_(x)     # no 16-byte pieces
        want = F.flashopt_mx_product(F.flashopt_mx_quantize(x), w)
        assert torch.equal(F.flashopt_mx_linear(x, w), want), m
        assert torch.equal(F.flashopt_mx_linear(apart, w), want), m


@pytest.mark.parametrize("m,n,k", [(5, 40, 130), (20, 9000, 130), (64, 64, 130), (300, 1100, 130), (300, 1100, 384),
                                   (300, 1100, 6017), (2000, 1800, 130), (3600, 3900, 130)])
@pytest.mark.parametrize("far", [254, 0])
def test_product_at_the_last_scales(m, n, k, far):
    """Scales 2^127 against 2^-127, whose values alone pass fp32's ends, and
    the zeros beside them (codes, padding, the absent half of a K step): a
    product of 1 times small multiples of 1/4, exact in any order."""
    require_gpu()
    g = torch.Generator().manual_seed(m + k)
    blocks = (k + 127) // 128
    there = torch.arange(128 * blocks) < k

    def one(rows, byte):
        codes = torch.randint(0, 256, (rows, 64 * blocks), generator=g, dtype=torch.uint8)
        codes = torch.where(there[0::2], codes & 15, 0) | torch.where(there[1::2], codes >> 4 << 4, 0)
        scales = torch.where(torch.arange(4 * blocks) * 32 < k, byte, 0).expand(rows, -1)
        return codes.to(torch.uint8).cuda(), scales.to(torch.uint8).cuda().contiguous()

    def values(codes):
        table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device="cuda")
        table = torch.cat([table, -table])
        return torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], 2).flatten(1)
    (ca, sa), (cb, sb) = one(m, far), one(n, 254 - far)
    want = values(ca) @ values(cb).t()
    print(f"{m} x {n} x {k}, A's scales {far}", flush=True)
    out = F.flashopt_mx_product(F.MXTensor(ca, sa, m, k), F.MXTensor(cb, sb, n, k), torch.float32)
    assert torch.equal(out.double(), want)
