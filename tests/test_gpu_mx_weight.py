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
