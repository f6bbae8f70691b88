"""mx_linear's calls, without a GPU: which copies are made for which
gradients.  The library's calls are replaced by ones that count."""
import contextlib

import pytest
import torch

from bit_companded_adam_amd import flashopt as F


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def quantize(x, layout="rows", out=None, stream=None):
        seen.append(layout)
        q = F.MXTensor.empty(*x.shape, "cpu")
        t = F.MXTensor.empty(*x.shape[::-1], "cpu")
        return (q, t) if layout == "both" else q if layout == "rows" else t

    def product(a, b, dtype=torch.bfloat16, out=None, stream=None):
        seen.append("product")
        return torch.zeros(a.rows, b.rows, dtype=dtype)
    monkeypatch.setattr(F, "flashopt_mx_quantize", quantize)
    monkeypatch.setattr(F, "flashopt_mx_product", product)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_transposed_without_gradients(calls, off):
    """Parameters require gradients in an evaluation too; with the gradients
    off, neither operand is quantized for a backward pass."""
    x, w = torch.zeros(4, 64, requires_grad=True), torch.zeros(3, 64, requires_grad=True)
    with off():
        y = F.mx_linear(x, w)
    assert y.shape == (4, 3) and calls == ["rows", "rows", "product"]
    del calls[:]
    held = F.MXWeight(w)
    assert calls.pop() == "both"
    with off():
        F.mx_linear(x, held)
    assert calls == ["rows", "product"]


def test_copies_follow_the_gradients_asked_for(calls):
    for need_x, need_w, want in ((True, True, ["both", "both"]), (True, False, ["both", "rows"]),
                                 (False, True, ["rows", "both"]), (False, False, ["rows", "rows"])):
        x, w = torch.zeros(4, 64, requires_grad=need_x), torch.zeros(3, 64, requires_grad=need_w)
        F.mx_linear(x, w)
        assert calls == want + ["product"]               # the weight first, then x
        del calls[:]
        with contextlib.nullcontext() if need_x or need_w else pytest.raises(RuntimeError):
            F.mx_linear(x, w).sum().backward()
        del calls[:]
