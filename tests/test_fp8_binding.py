"""fp8_linear's, rms_norm's and fp8_norm_linear's calls, without a GPU: which
copies are made for which gradients.  The library's calls are replaced by ones
that count."""
import contextlib

import pytest
import torch

from bit_companded_adam_amd import flashopt as F

E5M2 = torch.float8_e5m2


@pytest.fixture
def calls(monkeypatch):
    seen = []

    def made(rows, cols, layout, dtype=torch.float8_e4m3fn):
        q, t = F.FP8Tensor.empty(rows, cols, "cpu", dtype), F.FP8Tensor.empty(cols, rows, "cpu", dtype)
        return (q, t) if layout == "both" else q if layout == "rows" else t

    def quantize(x, layout="rows", block=False, dtype=torch.float8_e4m3fn, out=None, stream=None):
        seen.append(layout + (", block" if block else "") + (", e5m2" if dtype == E5M2 else ""))
        return made(*x.shape, layout, dtype)

    def product(a, b, dtype=torch.bfloat16, out=None, stream=None):
        seen.append("product")
        assert a.cols == b.cols
        return torch.zeros(a.rows, b.rows, dtype=dtype)

    def norm(x, gain, residual=None, eps=1e-6, output="values", dtype=torch.float8_e4m3fn, out=None, h=None,
             rstd=None, stream=None):
        seen.append("norm " + output)
        h = x if residual is None else x + residual
        return torch.zeros_like(x) if output == "values" else made(*x.shape, output), h

    def backward(dy, h, gain, rstd, dh=None, need_dx=True, need_dgain=True, **_):
        seen.append("backward" + " dx" * need_dx + " dgain" * need_dgain + " dh" * (dh is not None))
        return torch.zeros_like(h) if need_dx else None, torch.zeros_like(gain) if need_dgain else None
    monkeypatch.setattr(F, "flashopt_byte_quantize", quantize)
    monkeypatch.setattr(F, "flashopt_byte_product", product)
    monkeypatch.setattr(F, "flashopt_rms_norm", norm)
    monkeypatch.setattr(F, "flashopt_rms_norm_backward", backward)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return seen


@pytest.mark.parametrize("off", [torch.no_grad, torch.inference_mode])
def test_nothing_is_transposed_without_gradients(calls, off):
    x, w = torch.zeros(4, 64, requires_grad=True), torch.zeros(3, 64, requires_grad=True)
    gain = torch.zeros(64, requires_grad=True)
    with off():
        assert F.fp8_linear(x, w).shape == (4, 3)
    assert calls == ["rows, block", "rows", "product"]
    del calls[:]
    held = F.FP8Weight(w)
    assert calls.pop() == "both, block"
    with off():
        F.fp8_linear(x, held)
        F.fp8_norm_linear(x, gain, held)
        F.fp8_norm_linear(x, gain, w, x)
    assert calls == ["rows", "product", "norm rows", "product", "rows, block", "norm rows", "product"]


def test_linear_copies_follow_the_gradients_asked_for(calls):
    for need_x, need_w, want, back in (
            (True, True, ["both, block", "both"], ["both, e5m2", "product", "product"]),
            (True, False, ["both, block", "rows"], ["rows, e5m2", "product"]),
            (False, True, ["rows, block", "both"], ["cols, e5m2", "product"]),
            (False, False, ["rows, block", "rows"], None)):
        x, w = torch.zeros(4, 64, requires_grad=need_x), torch.zeros(3, 64, requires_grad=need_w)
        y = F.fp8_linear(x, w, grad_dtype=E5M2)
        assert calls == want + ["product"]               # the weight first, then x
        del calls[:]
        with contextlib.nullcontext() if back else pytest.raises(RuntimeError):
            y.sum().backward()
        assert calls == (back or [])
        del calls[:]


def test_norm_linear_copies_follow_the_gradients_asked_for(calls):
    for need_x, need_gain, need_w, need_res, weight, norm, back in (
            (1, 1, 1, 1, "both", "both", ["both", "product", "product", "backward dx dgain"]),
            (0, 0, 0, 1, "both", "rows", ["rows", "product", "backward dx"]),
            (0, 1, 0, 0, "both", "rows", ["rows", "product", "backward dgain"]),
            (0, 0, 1, 0, "rows", "both", ["cols", "product"]),
            (0, 1, 1, 0, "both", "both", ["both", "product", "product", "backward dgain"])):
        x, gain = torch.zeros(4, 64, requires_grad=bool(need_x)), torch.zeros(64, requires_grad=bool(need_gain))
        w, res = torch.zeros(3, 64, requires_grad=bool(need_w)), torch.zeros(4, 64, requires_grad=bool(need_res))
        for use_h in (False, True):
            y, h = F.fp8_norm_linear(x, gain, w, res)
            assert calls == [weight + ", block", "norm " + norm, "product"]
            del calls[:]
            ((y.sum() + h.sum()) if use_h else y.sum()).backward()
            assert calls == [c + " dh" if use_h and c.startswith("backward") else c for c in back]
            del calls[:]
        y, h = F.fp8_norm_linear(x, gain, w, res)
        del calls[:]
        h.sum().backward()                               # the sum alone: nothing to compute
        assert calls == []


def test_buffers_are_released_with_the_graph(calls):
    """What a forward pass keeps goes when its backward pass has run."""
    import gc
    import weakref
    x, gain = torch.zeros(4, 64, requires_grad=True), torch.zeros(64, requires_grad=True)
    w = torch.zeros(3, 64, requires_grad=True)
    for layer in (lambda: F.fp8_linear(x, w), lambda: F.fp8_norm_linear(x, gain, w)[0]):
        y = layer()
        kept = [weakref.ref(t) for t in y.grad_fn.saved_tensors if t.dtype == torch.uint8]
        assert len(kept) == 2
        y.sum().backward()
        gc.collect()
        assert all(k() is None for k in kept)


def test_matrices_of_another_layout_are_refused():
    """An 8-bit matrix has fewer bytes of scales than the 4-bit calls read, and
    the reverse of codes."""
    eight, four = F.FP8Tensor.empty(8, 4096, "cpu"), F.MXTensor.empty(8, 4096, "cpu")
    x = torch.zeros(2, 4096)
    for call in (lambda: F.flashopt_mx_product(eight, four), lambda: F.flashopt_mx_product(four, eight),
                 lambda: F.flashopt_mx_dequantize(eight), lambda: F.flashopt_mx_linear(x, eight),
                 lambda: F._mx_target(eight, 8, 4096, torch.device("cpu"))):
        with pytest.raises(ValueError, match="must be an MXTensor, got FP8Tensor"):
            call()
    for call in (lambda: F.flashopt_byte_product(eight, four), lambda: F.flashopt_byte_product(four, eight),
                 lambda: F.flashopt_byte_dequantize(four), lambda: F.flashopt_byte_linear(x, four),
                 lambda: F._fp8_target(four, 8, 4096, torch.device("cpu"), torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match="must be an FP8Tensor, got MXTensor"):
            call()
    for call in (lambda: F.mx_linear(x, F.FP8Weight.__new__(F.FP8Weight)),
                 lambda: F.fp8_linear(x, F.MXWeight.__new__(F.MXWeight))):
        with pytest.raises(ValueError, match="weight must be"):
            call()


def test_gradients_of_too_many_columns_are_refused_in_the_forward_call(calls):
    cols = F.NORM_GRAD_COLS + 1
    plain = dict(x=torch.zeros(2, cols), gain=torch.ones(cols), residual=torch.zeros(2, cols))
    w = torch.zeros(3, cols, requires_grad=True)
    for name in plain:
        args = {k: t.clone().requires_grad_(k == name) for k, t in plain.items()}
        for call in (lambda: F.rms_norm(**args), lambda: F.fp8_norm_linear(weight=w, **args)):
            with pytest.raises(ValueError, match="gradients have at most 32768"):
                call()
        with torch.no_grad():
            F.rms_norm(**args), F.fp8_norm_linear(weight=w, **args)
    F.rms_norm(**plain)
    F.fp8_norm_linear(weight=w, **plain)[0].sum().backward()        # the weight's gradient has no such bound
    assert w.grad.shape == w.shape and calls[-1] == "product"
    x = torch.zeros(2, cols - 1, requires_grad=True)
    F.rms_norm(x, torch.ones(cols - 1))[0].sum().backward()


def test_a_second_derivative_is_refused(calls):
    x, w, gain = (torch.ones(*s, requires_grad=True) for s in ((4, 64), (3, 64), (64,)))
    for out in (F.fp8_linear(x, w), F.rms_norm(x, gain)[0], F.fp8_norm_linear(x, gain, w)[0]):
        loss = out.square().sum()                 # whose gradient depends on out
        g, = torch.autograd.grad(loss, x, create_graph=True, retain_graph=False)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            g.sum().backward()
        with pytest.raises(RuntimeError, match="second time"):      # the first graph was used up
            loss.backward()
