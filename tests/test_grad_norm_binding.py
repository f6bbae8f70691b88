"""The binding's side of the gradient norm, without a GPU."""
import threading

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
