"""What rms_norm and fp8_norm_linear keep for their backward passes, without a
GPU: only what the gradients asked for read, so that nothing else is held in
memory, and a change of it refuses no backward pass that does not need it."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests.test_fp8_binding import calls  # noqa: F401


def _leaves(need, shape=(4, 64)):
    return [torch.zeros(s, requires_grad=n) for s, n in zip((shape, (64,), (3, 64), shape), need)]


def _refresh(weight):
    """As the library's call into the held copies counts."""
    weight.version += 1
    weight.rows._written(), weight.cols._written()


def test_the_sum_alone_reads_nothing(calls):  # noqa: F811
    """A loss of h alone: neither the gain, h, the weight's copies nor the
    activation's are read, whatever has happened to them."""
    for held in (False, True):
        x, gain, w, res = _leaves((True,) * 4)
        weight = F.FP8Weight(w) if held else w
        for layer in (lambda: F.rms_norm(x, gain, res), lambda: F.fp8_norm_linear(x, gain, weight, res)):
            y, h = layer()
            with torch.no_grad():
                gain.add_(1), h.add_(1), w.add_(1)
            if held:
                _refresh(weight)
            h.sum().backward()
            assert torch.equal(x.grad, torch.ones(4, 64)) and torch.equal(res.grad, x.grad) and gain.grad is None
            x.grad = res.grad = None


def test_the_weight_alone_needs_no_norm(calls):  # noqa: F811
    """Frozen inputs and gain: the weight's gradient reads the activation's
    8-bit columns only."""
    for residual in (False, True):
        x, gain, w, res = _leaves((False, False, True, False))
        y, h = F.fp8_norm_linear(x, gain, w, res if residual else None)
        assert [t.dtype for t in y.grad_fn.saved_tensors] == [torch.uint8]
        with torch.no_grad():
            gain.add_(1), h.add_(1)
        y.sum().backward()
        assert w.grad is not None and not any(c.startswith("backward") for c in calls)


def test_what_is_read_is_kept(calls):  # noqa: F811
    for need in ((1, 0, 0, 0), (0, 1, 0, 0), (0, 0, 0, 1), (1, 1, 1, 1)):
        x, gain, w, res = _leaves(map(bool, need))
        y, h = F.fp8_norm_linear(x, gain, w, res)
        assert [t.dtype for t in y.grad_fn.saved_tensors].count(torch.float32) == 3      # h, the gain and 1 / root
        with torch.no_grad():
            gain.add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.sum().backward()


def test_a_refresh_between_the_passes_is_named(calls):  # noqa: F811
    for need in ((1, 0, 0, 0), (0, 1, 1, 0)):
        x, gain, w, res = _leaves(map(bool, need))
        weight = F.FP8Weight(w)
        y, _ = F.fp8_norm_linear(x, gain, weight, res)
        _refresh(weight)
        with pytest.raises(RuntimeError, match="FP8Weight was refreshed"):
            y.sum().backward()
    x, gain, w, res = _leaves((False, False, True, False))
    weight = F.FP8Weight(w)
    y, _ = F.fp8_norm_linear(x, gain, weight, res)
    _refresh(weight)
    y.sum().backward()                            # reads no copy of the weight
    assert w.grad is not None
