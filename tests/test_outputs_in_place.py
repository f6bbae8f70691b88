"""In-place work on the outputs of mx_linear, fp8_linear, rms_norm and
fp8_norm_linear, without a GPU: an output is a tensor of its own, as that of
torch's own layers, whatever the number of dimensions."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests.test_fp8_binding import calls  # noqa: F401
from tests.test_mx_binding import calls as mx_calls  # noqa: F401

SHAPES = [(64,), (4, 64), (2, 3, 64), (2, 0, 64), (2, 2, 3, 64)]


def _leaves(shape):
    return [torch.ones(s, requires_grad=True) for s in (shape, (64,), (5, 64), shape)]


def _check(y, x, shape):
    assert y.shape == shape and not y._is_view() and y.requires_grad
    y += 1
    y.mul_(2)
    torch.relu_(y)
    y.sum().backward()
    assert x.grad.shape == x.shape


@pytest.mark.parametrize("shape", SHAPES)
def test_linear(calls, mx_calls, shape):  # noqa: F811
    for layer in (F.fp8_linear, F.mx_linear):
        x, _, w, _ = _leaves(shape)
        _check(layer(x, w), x, (*shape[:-1], 5))
        x.grad = None
        y = layer(x, w)
        y.view(-1)[:3].zero_()              # a view of it, too
        y.sum().backward()
        with torch.no_grad():
            layer(x, w).mul_(2)


@pytest.mark.parametrize("shape", SHAPES)
def test_norm(calls, shape):  # noqa: F811
    x, gain, _, res = _leaves(shape)
    _check(F.rms_norm(x, gain)[0], x, shape)
    x.grad = None
    y, h = F.rms_norm(x, gain, res)
    assert not h._is_view()
    _check(y, x, shape)
    assert torch.equal(res.grad, x.grad)


@pytest.mark.parametrize("shape", SHAPES)
def test_norm_linear(calls, shape):  # noqa: F811
    for residual in (False, True):
        x, gain, w, res = _leaves(shape)
        y, h = F.fp8_norm_linear(x, gain, w, res if residual else None)
        assert not h._is_view()
        _check(y, x, (*shape[:-1], 5))
        assert torch.equal(w.grad, torch.zeros(5, 64)) and (not residual or torch.equal(res.grad, x.grad))


@pytest.mark.parametrize("shape", SHAPES)
def test_the_sum(calls, shape):  # noqa: F811
    """h may be changed in place; a backward pass that reads it says so."""
    for layer in (lambda: F.rms_norm(x, gain, res), lambda: F.fp8_norm_linear(x, gain, w, res)):
        x, gain, w, res = _leaves(shape)
        y, h = layer()
        h += 1
        assert h.shape == shape and torch.equal(h, torch.full(shape, 3.0))
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()
