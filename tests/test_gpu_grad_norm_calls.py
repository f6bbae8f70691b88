"""Norm and clipping called in the less usual ways: with the caller's own
workspace under capture, and from several host threads at once."""
import ctypes
import threading

import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
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


def test_threads_on_one_stream():
    """Norms and clips of lists of different lengths, each with its table in
    a workspace, from several host threads on the default stream: every thread
    sees its own list."""
    require_gpu()
    sizes = (70, 201, 90, 3, 130)
    lists = [[W.make_grad(500 + 37 * i, k, device="cuda", stream_id=i) for i in range(n)]
             for k, n in enumerate(sizes)]
    copies = [[g.clone() for g in grads] for grads in lists]
    bounds = [0.9 ** (i + 1) * float(F.flashopt_grad_norm(lists[0])[0]) for i in range(12)]

    def run(grads):                      # norm and clip in turn, every clip scaling
        out = []
        for bound in bounds:
            out += [F.flashopt_grad_norm(grads, bound), F.flashopt_grad_clip(grads, bound)]
        return out
    want = [run(grads) for grads in copies]
    torch.cuda.synchronize()
    got, errors = [None] * len(lists), []
    start = threading.Barrier(len(lists))

    def work(k):
        try:
            start.wait(30)
            got[k] = run(lists[k])
        except Exception as e:           # raised again below
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(lists))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for k in range(len(lists)):
        assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), k
        # the three tensors' norm, a ninth of the first list's, is below the last bound, 0.28 of it
        assert (float(got[k][-1][1]) < 1.0) == (sizes[k] > 3)
        assert all(torch.equal(a, b) for a, b in zip(lists[k], copies[k])), k
