"""Batches without rows through every layer, forward and backward, with the
gradients that autograd makes of a plain sum (strides of 0 throughout)."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import _random

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("shape", [(0, 64), (3, 0, 64), (0, 5, 64), (2, 0, 3, 64)])
@pytest.mark.parametrize("layer", ["mx_linear", "fp8_linear", "rms_norm", "fp8_norm_linear"])
def test_no_rows(layer, shape):
    require_gpu()
    for residual in (False, True):
        x, res = (torch.zeros(shape, dtype=BF16, device="cuda", requires_grad=True) for _ in range(2))
        gain, w = _random(64, 1, BF16).requires_grad_(), _random((40, 64), 2, BF16).requires_grad_()
        r = res if residual else None
        outs = {"mx_linear": lambda: (F.mx_linear(x, w),), "fp8_linear": lambda: (F.fp8_linear(x, w),),
                "rms_norm": lambda: F.rms_norm(x, gain, r),
                "fp8_norm_linear": lambda: F.fp8_norm_linear(x, gain, w, r, norm_grad_dtype=torch.float32)}[layer]()
        assert outs[0].shape == (*shape[:-1], 40 if "linear" in layer else 64)
        sum(o.float().sum() for o in outs).backward()
        assert x.grad.shape == shape
        used = {"mx_linear": (w,), "fp8_linear": (w,), "rms_norm": (gain,), "fp8_norm_linear": (w, gain)}[layer]
        for t in used:
            assert torch.equal(t.grad, torch.zeros_like(t))


def test_raw_calls_of_empty_expanded_matrices():
    require_gpu()
    z = torch.ones(1, 1, dtype=BF16, device="cuda").expand(0, 64)
    assert z.stride(1) == 0
    gain, rstd = _random(64, 1, BF16), torch.empty(0, device="cuda")
    y, h = F.flashopt_rms_norm(z, gain, z)
    assert y.shape == h.shape == (0, 64)
    dx, dgain = F.flashopt_rms_norm_backward(z, z, gain, rstd, z)
    assert dx.shape == (0, 64) and torch.equal(dgain, torch.zeros_like(gain))
    for quantize in (F.flashopt_byte_quantize, F.flashopt_mx_quantize):
        q, t = quantize(z, "both")
        assert (q.rows, q.cols, t.rows, t.cols) == (0, 64, 64, 0)
    full = torch.ones(1, 1, dtype=BF16, device="cuda").expand(2, 64)       # rows there are: still refused
    with pytest.raises(ValueError, match="rows must be contiguous"):
        F.flashopt_byte_quantize(full)
    with pytest.raises(ValueError, match="rows must be contiguous"):
        F.flashopt_rms_norm(torch.ones(2, 64, dtype=BF16, device="cuda"), gain, full)
