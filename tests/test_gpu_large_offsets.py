"""Sizes past 32 bits: gradients of more than 2^32 elements or 8 GB, and
weights of more rows than one pass of the few-row product's grid takes."""
import math

import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
HALF = 2.0 ** -24 * (1 + 2.0 ** -20)      # one fp32 rounding, over the fp64 error of so few terms


@pytest.mark.parametrize("dtype,n", [(BF16, (1 << 32) + 12345), (F32, (1 << 31) + 12345)])
def test_norm_and_clip_past_32_bits(dtype, n):
    """Zeros but for values on both sides of 2^30, 2^31 and 2^32 elements and
    at the ends, in a view that starts at an odd element, between two small
    gradients; what lies around the view stays."""
    require_gpu()
    flat = torch.zeros(n + 4, dtype=dtype, device="cuda")
    flat[0], flat[-3:] = 7.0, 7.0
    big = flat[1:n + 1]
    at = sorted({i for e in (0, 1 << 30, 1 << 31, 1 << 32, n) for i in (e - 8193, e - 1, e, e + 1, e + 8191)
                 if 0 <= i < n})
    for k, i in enumerate(at):
        big[i] = float(k + 1)
    small = [torch.full((5,), 3.0, dtype=BF16, device="cuda"), torch.full((9001,), 0.5, device="cuda")]
    grads = [small[0], big, small[1]]
    print(f"{dtype} {n}", flush=True)
    norm = math.sqrt(sum((k + 1) ** 2 for k in range(len(at))) + 5 * 9 + 9001 * 0.25)
    out = F.flashopt_grad_norm(grads, norm / 4).double().tolist()
    assert abs(out[0] - norm) <= HALF * norm
    out = F.flashopt_grad_clip(grads, norm / 4)
    scale = norm / 4 / (norm + 1e-6)
    assert abs(float(out[1]) - scale) <= HALF * scale
    want = (torch.arange(1, len(at) + 1, device="cuda").float() * out[1]).to(dtype)
    got = torch.stack([big[i] for i in at])
    assert torch.equal(got, want)
    for i in at:
        big[i] = 0.0
    bits = big.view(torch.int16 if dtype == BF16 else torch.int32)
    assert not any(bool(part.any()) for part in bits.split(1 << 30))
    assert flat[0] == 7.0 and (flat[-3:] == 7.0).all()
    for g, value in ((small[0], 3.0), (small[1], 0.5)):
        assert (g == (torch.tensor(value, device="cuda") * out[1]).to(g.dtype)).all()


@pytest.mark.parametrize("m,n", [(1, (1 << 25) + 100_003), (5, (1 << 26) + 70_001)])
def test_few_rows_over_more_weights_than_one_grid(m, n):
    """2^20 workgroups of 32 or 64 rows of the weight, and some that take a
    second tile: exact (small integers times 1/4: every sum is)."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(m)
    codes = torch.zeros(n, 64, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(n, 4, dtype=torch.uint8, device="cuda")
    part = 1 << 22
    for i in range(0, n, part):
        rows = min(part, n - i)
        codes[i:i + rows, :16] = torch.randint(0, 256, (rows, 16), generator=g, device="cuda", dtype=torch.uint8)
        scales[i:i + rows, 0] = torch.randint(126, 129, (rows,), generator=g, device="cuda", dtype=torch.uint8)
    w = F.MXTensor(codes, scales, n, 32)
    x = torch.randint(-3, 4, (m, 32), generator=g, device="cuda").float()
    a = F.flashopt_mx_quantize(x)
    assert torch.equal(F.flashopt_mx_dequantize(a), x)
    print(f"{m} x {n} x 32", flush=True)
    out = F.flashopt_mx_product(a, w, F32)
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    table = torch.cat([table, -table])
    for i in range(0, n, part):
        rows = min(part, n - i)
        c = codes[i:i + rows, :16].int()
        v = torch.stack([table[c & 15], table[c >> 4]], 2).view(rows, 32)
        v = v * torch.exp2(scales[i:i + rows, :1].float() - 127)
        want = torch.zeros(m, rows, device="cuda")
        for k in range(32):                              # sums of multiples of 1/4 below 2^11: exact in any order
            want += x[:, k:k + 1] * v[:, k]
        assert torch.equal(out[:, i:i + rows], want), i
