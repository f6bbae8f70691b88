"""Gradient release with a factor on the gradients (a loss scale's
reciprocal): the same bits as list steps with the same factor."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import require_gpu
from tests.test_gpu_grad_release import _assert_same

pytestmark = pytest.mark.gpu

SIZES = [1 << 17, 33, 70001, 5000]


@pytest.mark.parametrize("kind", ["adamw", "sgd"])
@pytest.mark.parametrize("batch_below,streams", [(65536, 4), (0, 1), (0, 3), (1 << 30, 2)])
def test_released_steps_are_scaled(kind, batch_below, streams):
    """Gradients that do not depend on the parameters, and a factor rewritten
    between backward passes."""
    require_gpu()
    make = (lambda p: F.FlashAdamW(p, **W.HP_DEFAULT)) if kind == "adamw" else (lambda p: F.FlashSGD(p, **W.SGD_DEFAULT))
    params = [W.init_param(n, device="cuda", seed=i).requires_grad_() for i, n in enumerate(SIZES)]
    other = [p.detach().clone() for p in params]
    a, b = make([p.detach() for p in params]), make(other)
    scale = torch.zeros(1, device="cuda")
    handles = F.attach_grad_release(a, params, batch_below=batch_below, streams=streams, grad_scale=scale)
    for t, factor in ((1, 2.0 ** -16), (2, 0.37), (3, 1.0)):
        grads = [W.make_grad(n, t, device="cuda", stream_id=i, scale=40.0) for i, n in enumerate(SIZES)]
        scale.fill_(factor)
        torch.autograd.backward(params, grads)
        assert all(p.grad is None for p in params)
        b.step(grads, grad_scale=torch.tensor([factor], device="cuda"))
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(a.states, b.states)):
            _assert_same(x, y, f"{kind} t{t} tensor{i}")
    for h in handles:
        h.remove()


def test_a_host_factor_is_refused():
    require_gpu()
    p = W.init_param(64, device="cuda").requires_grad_()
    with pytest.raises(ValueError, match="grad_scale"):
        F.attach_grad_release(F.FlashAdamW([p.detach()]), [p], grad_scale=torch.ones(1))
