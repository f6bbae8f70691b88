"""Norm and clipping called in the less usual ways: with the caller's own
workspace under capture, and from several host threads at once."""
import ctypes

import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu


def test_capture_of_a_long_list_with_a_workspace_is_refused():
    """The caller's workspace does not make a staged table capturable: the
    binding refuses the call, the library refuses it from C, and neither
    records anything.  A plan is not made in a capture either."""
    require_gpu()
    grads = [torch.full((8,), 2.0, device="cuda") for _ in range(65)]
    out = torch.zeros(2, device="cuda")
    ws = torch.zeros(F.flashopt_grad_workspace_bytes(65), dtype=torch.uint8, device="cuda")
    buf = torch.zeros(F.flashopt_grad_plan_bytes(65), dtype=torch.uint8, device="cuda")
    short = torch.zeros(F.flashopt_grad_workspace_bytes(64), dtype=torch.uint8, device="cuda")
    L, (arr, _) = F.lib(), F.grad_array(grads)
    info = F.flashopt_grad_plan_info(-1, -1, -1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (F.flashopt_grad_norm, F.flashopt_grad_clip):
            with pytest.raises(ValueError, match="GradPlan"):
                call(grads, 1.0, out=out, workspace=ws)
        with pytest.raises(ValueError, match="before the capture"):
            F.GradPlan(grads)
        stream = torch.cuda.current_stream().cuda_stream
        for call in (L.flashopt_grad_norm, L.flashopt_grad_clip):
            assert call(arr, 65, 1.0, out.data_ptr(), ws.data_ptr(), ws.numel(), stream) == F.FLASHOPT_EINVAL
        assert L.flashopt_grad_plan(arr, 65, buf.data_ptr(), buf.numel(), ctypes.byref(info), stream) == F.FLASHOPT_EINVAL
        F.flashopt_grad_norm(grads[:64], 1.0, out=out, workspace=short)
    assert info.n_tensors == -1
    for _ in range(3):
        out.zero_()
        graph.replay()
        again = F.flashopt_grad_norm(grads, 1.0, workspace=ws)        # eager work between the replays
        torch.cuda.synchronize()
        assert out[0].item() == float(torch.tensor(64 * 8 * 4.0).sqrt())
        assert again[0].item() == float(torch.tensor(65 * 8 * 4.0).sqrt())
    assert all((g == 2.0).all() for g in grads) and not buf.any()
