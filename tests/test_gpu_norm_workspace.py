"""The norm's backward pass writes its workspace's bytes and none behind them,
and a buffer made for a wider pass serves a narrower one."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import _random

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, 5), (1, 32768), (3, 1500), (5, 1000), (300, 2304), (700, 4096), (1200, 700),
                                       (2100, 64), (257, 16391)])
def test_what_lies_behind(rows, cols):
    require_gpu()
    h, dy, gain = (_random(s, i, torch.bfloat16) for i, s in enumerate(((rows, cols), (rows, cols), cols)))
    rstd = torch.ones(rows, device="cuda")
    want = F.flashopt_rms_norm_backward(dy, h, gain, rstd)
    for need in (F.flashopt_rms_norm_backward_workspace_bytes(rows, cols),
                 F.flashopt_rms_norm_backward_workspace_bytes(rows + 1, min(2 * cols, 32768))):
        whole = torch.full((need + 65536,), 77, dtype=torch.uint8, device="cuda")
        got = F.flashopt_rms_norm_backward(dy, h, gain, rstd, workspace=whole[:need])
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and (whole[need:] == 77).all()
