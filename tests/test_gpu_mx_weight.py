"""MXWeight between a forward and its backward pass: copies rewritten in
between are refused where the backward pass would read them, or were kept."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _random(rows, cols, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, cols, generator=g).to(BF16).cuda()


def test_refresh_does_not_touch_a_weight_gradient():
    """With no gradient to x (a first layer), backward reads no copy of the
    weight: a refresh in between changes nothing."""
    require_gpu()
    x, dy = _random(40, 100, 1), _random(40, 50, 2)
    w = _random(50, 100, 3).requires_grad_()
    weight = F.MXWeight(w)
    want = torch.autograd.grad(F.mx_linear(x, weight), w, dy)[0]
    y = F.mx_linear(x, weight)
    with torch.no_grad():
        w.mul_(2)
    weight.refresh()
    assert torch.equal(torch.autograd.grad(y, w, dy)[0], want)


def test_copies_rewritten_through_quantize_are_refused():
    """The copies written by another call than refresh(), in the MXWeight's own
    tensors or in others over the same memory."""
    require_gpu()
    x, dy = _random(40, 100, 1), _random(40, 50, 2)
    w = _random(50, 100, 3)
    weight = F.MXWeight(w)
    alias = F.MXTensor(weight.cols.codes, weight.cols.scales, 100, 50)
    for layout, out in (("both", (weight.rows, weight.cols)), ("cols", weight.cols), ("cols", alias)):
        y = F.mx_linear(x.clone().requires_grad_(), weight)
        F.flashopt_mx_quantize(w, layout, out)
        with pytest.raises(RuntimeError, match="modified"):
            y.backward(dy)
    y = F.mx_linear(x.clone().requires_grad_(), weight)
    F.flashopt_mx_quantize(w, out=weight.rows)               # which no backward pass reads
    y.backward(dy)
    with torch.inference_mode():                             # buffers without versions
        served = F.MXWeight(w)
        served.refresh()
        assert torch.equal(F.mx_linear(x, served), F.mx_linear(x, weight))
    served.refresh()
    assert torch.equal(served.rows.codes, weight.rows.codes)
