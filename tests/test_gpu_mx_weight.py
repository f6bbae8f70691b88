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


@pytest.mark.parametrize("how", ["refresh", "quantize"])
def test_replayed_refresh_between_forward_and_backward(how):
    """A replay rewrites the copies without the host's knowledge: an eager
    backward pass still multiplies by those of its own forward pass."""
    require_gpu()
    dy = _random(40, 50, 2)
    w = _random(50, 100, 3)
    weight = F.MXWeight(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if how == "refresh":
            weight.refresh()
        else:
            F.flashopt_mx_quantize(w, "both", (weight.rows, weight.cols))
    seen = []
    for i in range(4):
        w.copy_(_random(50, 100, 10 + i))
        graph.replay()
        x = _random(40, 100, 20 + i)
        a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
        want = torch.autograd.grad(F.mx_linear(a, w.clone()), a, dy)[0]
        y = F.mx_linear(b, weight)
        w.copy_(_random(50, 100, 30 + i))
        graph.replay()
        again = F.mx_linear(x, weight)
        y.backward(dy)
        torch.cuda.synchronize()
        assert torch.equal(b.grad, want), i
        assert torch.equal(again, F.mx_linear(x, w)) and not torch.equal(again, y), i
        seen.append(want)
    assert not torch.equal(seen[0], seen[1])


def test_weight_made_in_a_capture():
    """Its copies are the graph's, written by every replay."""
    require_gpu()
    dy, x = _random(40, 50, 2), _random(40, 100, 4)
    w = _random(50, 100, 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        weight = F.MXWeight(w)
    for i in range(3):
        w.copy_(_random(50, 100, 10 + i))
        graph.replay()
        a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
        want = torch.autograd.grad(F.mx_linear(a, w.clone()), a, dy)[0]
        y = F.mx_linear(b, weight)
        w.copy_(_random(50, 100, 30 + i))
        graph.replay()
        y.backward(dy)
        torch.cuda.synchronize()
        assert torch.equal(b.grad, want), i
