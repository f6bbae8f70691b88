"""In-place work on the layers' outputs on the GPU: the same values and
gradients as out of place, for rows and for batches of sequences."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import _random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(130,), (6, 130), (2, 3, 130)])
@pytest.mark.parametrize("layer", ["mx_linear", "fp8_linear", "rms_norm", "fp8_norm_linear"])
def test_in_place(layer, shape):
    require_gpu()
    x, res = _random(shape, 1, torch.bfloat16), _random(shape, 2, torch.bfloat16)
    gain, w = _random(130, 3, torch.bfloat16), _random((40, 130), 4, torch.bfloat16)

    def run(in_place):
        leaves = [t.clone().requires_grad_() for t in (x, gain, w, res)]
        a, g, b, r = leaves
        outs = {"mx_linear": lambda: (F.mx_linear(a, b),), "fp8_linear": lambda: (F.fp8_linear(a, b),),
                "rms_norm": lambda: F.rms_norm(a, g, r), "fp8_norm_linear": lambda: F.fp8_norm_linear(a, g, b, r)}[layer]()
        y = outs[0]
        y = torch.relu_(y.mul_(3)) if in_place else torch.relu(y * 3)
        sum(o.float().square().sum() for o in (y, *outs[1:])).backward()
        return [y.detach(), *[t.grad for t in leaves if t.grad is not None]]
    one, two = run(True), run(False)
    assert len(one) == len(two) and all(torch.equal(p, q) for p, q in zip(one, two))
