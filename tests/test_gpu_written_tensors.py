"""What a call writes into a tensor of the caller's counts as an in-place change
of it: a backward pass that has kept that tensor refuses, as after torch's own
in-place operations.  A call that is refused changes nothing."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import _random

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("shape", [(6, 64), (2, 3, 64)])
@pytest.mark.parametrize("place", ["h", "x", "out", "product", "linear", "dequantize", "dx"])
def test_the_sum_overwritten_between_the_passes(shape, place):
    require_gpu()
    x, res = _random(shape, 1, BF16).requires_grad_(), _random(shape, 2, BF16)
    gain, z = _random(64, 3, BF16).requires_grad_(), _random((6, 64), 4, BF16)
    w = F.flashopt_byte_quantize(_random((64, 64), 5, BF16))
    y, h = F.rms_norm(x, gain, res)
    y2, h2 = F.fp8_norm_linear(x, gain, _random((32, 64), 6, BF16), res)
    for out, kept in ((y, h), (y2, h2)):
        flat, g = kept.detach().view(-1, 64), gain.detach()
        before = flat.clone()
        if place == "h":
            F.flashopt_rms_norm(z, g, flat, h=flat)
        elif place == "x":
            F.flashopt_rms_norm(flat, g, z, h=flat)
        elif place == "out":
            F.flashopt_rms_norm(z, g, out=flat)
        elif place == "product":
            F.flashopt_byte_product(F.flashopt_byte_quantize(z), w, out=flat)
        elif place == "linear":
            F.flashopt_byte_linear(z, w, out=flat)
        elif place == "dequantize":
            F.flashopt_byte_dequantize(F.flashopt_byte_quantize(z), out=flat)
        else:
            F.flashopt_rms_norm_backward(z, z, g, torch.ones(6, device="cuda"), dx=flat)
        assert not torch.equal(flat, before)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.sum().backward()


def test_the_four_bit_calls_too():
    require_gpu()
    z, q = _random((6, 64), 1, BF16), F.flashopt_mx_quantize(_random((64, 64), 2, BF16))
    for call in (lambda out: F.flashopt_mx_product(F.flashopt_mx_quantize(z), q, out=out),
                 lambda out: F.flashopt_mx_linear(z, q, out=out),
                 lambda out: F.flashopt_mx_dequantize(F.flashopt_mx_quantize(z), out=out)):
        a, b = _random((6, 64), 3, BF16).requires_grad_(), _random((6, 64), 4, BF16)
        c = a * b
        call(b)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            c.sum().backward()


def _versions(*tensors):
    return [t._version for t in tensors]


def test_every_output_is_counted():
    require_gpu()
    x, gain, h, out = _random((5, 40), 1, F32), _random(40, 2, BF16), _random((5, 40), 3, F32), torch.empty(5, 40, device="cuda")
    rstd, dx, dgain = torch.empty(5, device="cuda"), torch.empty(5, 40, device="cuda"), torch.empty_like(gain)
    inputs = _versions(x, gain)
    before = _versions(h, out, rstd)
    F.flashopt_rms_norm(x, gain, x, out=out, h=h, rstd=rstd)
    assert all(b > a for a, b in zip(before, _versions(h, out, rstd)))
    q = F.flashopt_byte_quantize(x)
    before = _versions(h, out, rstd)
    F.flashopt_rms_norm(x, gain, x, h=h, rstd=rstd, output="rows", out=q)
    after = _versions(h, out, rstd)
    assert after[0] > before[0] and after[1] == before[1] and after[2] > before[2]
    before = _versions(dx, dgain, rstd, h)
    F.flashopt_rms_norm_backward(x, h, gain, rstd, dx=dx, dgain=dgain)
    after = _versions(dx, dgain, rstd, h)
    assert after[0] > before[0] and after[1] > before[1] and after[2:] == before[2:]
    assert _versions(x, gain) == inputs


def test_refused_calls_count_nothing():
    require_gpu()
    x, gain, y = _random((5, 40), 1, F32), _random(40, 2, BF16), torch.empty(5, 41, device="cuda")
    rstd = torch.ones(5, device="cuda")
    before = _versions(x, gain, y, rstd)
    for call in (lambda: F.flashopt_rms_norm(x, gain, out=x), lambda: F.flashopt_rms_norm(x, gain, x.clone(), out=x),
                 lambda: F.flashopt_rms_norm_backward(x, x, gain, rstd, dx=x),
                 lambda: F.flashopt_rms_norm(x, gain, rstd=rstd, eps=-1.0),
                 lambda: F.flashopt_byte_product(F.flashopt_byte_quantize(x), F.flashopt_byte_quantize(x), out=y),
                 lambda: F.flashopt_byte_dequantize(F.flashopt_byte_quantize(x), out=y)):
        with pytest.raises((F.FlashoptError, ValueError)):
            call()
    assert _versions(x, gain, y, rstd) == before


def test_tensors_of_inference_mode():
    """They have no versions and no backward pass: written in and out of it."""
    require_gpu()
    x, gain = _random((5, 40), 1, F32), _random(40, 2, F32)
    want, _ = F.flashopt_rms_norm(x, gain)
    with torch.inference_mode():
        y = torch.empty(5, 40, device="cuda")
        F.flashopt_rms_norm(x, gain, out=y)
        assert torch.equal(y, want)
    y.data.zero_()
    F.flashopt_rms_norm(x, gain, out=y)
    assert torch.equal(y, want)
