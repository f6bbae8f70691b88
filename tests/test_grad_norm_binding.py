"""The binding's side of the gradient norm, without a GPU."""
import threading

import pytest
import torch

from bit_companded_adam_amd import flashopt as F


def test_a_workspace_belongs_to_one_host_thread(monkeypatch):
    """Threads on one stream: a long list's call copies its table and then
    launches, so another thread's table must not land in the same workspace."""
    monkeypatch.setattr(F, "_stream", lambda stream: 7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    device, got = torch.device("cpu"), {}

    def work(name):
        first = F._grad_workspace(70, device)
        got[name] = (first, F._grad_workspace(70, device), F._grad_workspace(3, device))
    work("main")
    threads = [threading.Thread(target=work, args=(k,)) for k in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for first, again, short in got.values():
        assert first is again and first is short            # kept from call to call
    assert len({ws[0].data_ptr() for ws in got.values()}) == 4
    grown = F._grad_workspace(5000, device)
    assert grown.numel() >= F.flashopt_grad_workspace_bytes(5000) and not grown.any()


@pytest.mark.parametrize("call", [lambda g: F.flashopt_grad_norm(g), lambda g: F.flashopt_grad_clip(g, 1.0),
                                  lambda g: F.GradPlan(g)])
def test_a_missing_gradient_is_named(call):
    """Parameters that took no part in the loss have a .grad of None."""
    with pytest.raises(ValueError, match="gradient 1 is None"):
        call([torch.zeros(8), None, torch.zeros(3)])
