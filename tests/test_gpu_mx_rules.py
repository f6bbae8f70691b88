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
