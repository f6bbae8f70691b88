"""The norm's backward pass with an fp32 gradient of a bf16 norm, and
fp8_norm_linear, whose product can hand it over unrounded.  Against the formula
in 64 bits, with a bound for each fp32 operation."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import COLS, U, _backward, _check_backward, _half, _random

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _norm_inputs(rows, cols, seed=0):
    h, gain = _random((rows, cols), seed + 1, BF16, 2.0), _random(cols, seed + 2, BF16)
    dy, dh = _random((rows, cols), seed + 3, F32, 1e-3), _random((rows, cols), seed + 4, BF16, 1e-3)
    rstd = torch.empty(rows, device="cuda")
    F.flashopt_rms_norm(h, gain, rstd=rstd)
    return dy, h, gain, rstd, dh


@pytest.mark.parametrize("cols", [c for c in COLS if c <= 32768])
def test_backward_of_an_fp32_gradient(cols):
    """Every width's kernel; the same values in bf16 give the same bits."""
    require_gpu()
    for rows in (1, 3, 33, 130, 1100):
        if rows * cols > 5_000_000:
            continue
        dy, h, gain, rstd, dh = _norm_inputs(rows, cols, cols + rows)
        dh = dh if rows != 3 else None
        dx, dgain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh)
        assert dx.dtype == dgain.dtype == BF16
        _check_backward(dx, dgain, dy, h, gain, rstd, dh)
        only_x, _ = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh, need_dgain=False)
        _, only_gain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh, need_dx=False)
        assert torch.equal(only_x, dx) and torch.equal(only_gain, dgain)
        short = dy.to(BF16)
        for a, b in zip(F.flashopt_rms_norm_backward(short, h, gain, rstd, dh),
                        F.flashopt_rms_norm_backward(short.float(), h, gain, rstd, dh)):
            assert torch.equal(a, b)
        if dh is not None:
            over = dh.clone()
            F.flashopt_rms_norm_backward(dy, h, gain, rstd, over, dx=over)
            assert torch.equal(over, dx)


def test_views_of_an_fp32_gradient():
    """Row strides and odd offsets, a gradient that repeats one row, and the
    refusal of dx over it."""
    require_gpu()
    for cols in (41, 1300, 5001):
        dy, h, gain, rstd, dh = _norm_inputs(70, cols)
        want = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh)
        wide = _random((70, cols + 7), 9, F32)
        wide[:, 3:cols + 3] = dy
        around = wide.clone()
        got = F.flashopt_rms_norm_backward(wide[:, 3:cols + 3], h, gain, rstd, dh)
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(wide, around)
        row = dy[:1].expand(70, cols)
        for a, b in zip(F.flashopt_rms_norm_backward(row, h, gain, rstd, dh),
                        F.flashopt_rms_norm_backward(row.contiguous(), h, gain, rstd, dh)):
            assert torch.equal(a, b)
        with pytest.raises(F.FlashoptError):
            F.flashopt_rms_norm_backward(dy, h, gain, rstd, dx=dy.view(BF16)[:, :cols])
        with pytest.raises(ValueError, match="dy must be"):
            F.flashopt_rms_norm_backward(dy.half(), h, gain, rstd)
        with pytest.raises(ValueError, match="dy must be"):      # bf16 beside fp32 is no choice
            F.flashopt_rms_norm_backward(dy.to(BF16), h.float(), gain, rstd)


@pytest.mark.parametrize("kind", [E4M3, E5M2])
@pytest.mark.parametrize("shape,n", [((1, 40), 30), ((2, 50, 300), 129), ((300, 2048), 700)])
def test_norm_linear_gradients_in_one_rounding(shape, n, kind):
    """With norm_grad_dtype=float32 dx and dgain are the fp32 product's values
    taken through the norm's backward pass and rounded to bf16 once, at its end;
    by default, twice.  Outputs and the weight's gradient are the same."""
    require_gpu()
    k = shape[-1]
    x, gain, res = _random(shape, 1, BF16), _random(k, 2, BF16), _random(shape, 3, BF16)
    w, dy, dh = _random((n, k), 4, BF16, 0.1), _random((*shape[:-1], n), 5, BF16, 1e-3), _random(shape, 6, BF16, 1e-3)
    rows = x.numel() // k
    rstd = torch.empty(rows, device="cuda")
    _, h0 = F.flashopt_rms_norm(x.view(-1, k), gain, res.view(-1, k), rstd=rstd)
    _, w_cols = F.flashopt_byte_quantize(w, "both", block=True)
    dn = F.flashopt_byte_product(F.flashopt_byte_quantize(dy.view(-1, n), dtype=kind), w_cols, F32)
    grads = {}
    for choice in (F32, BF16, None):
        leaves = [t.clone().requires_grad_() for t in (x, gain, w, res)]
        outs = F.fp8_norm_linear(*leaves, grad_dtype=kind, norm_grad_dtype=choice)
        grads[choice] = (*outs, *torch.autograd.grad(outs, leaves, (dy, dh)))
    y, h, dx, dgain, dw, dres = grads[F32]
    _check_backward(dx.view(-1, k), dgain, dn, h0, gain, rstd, dh.view(-1, k))
    want = F.flashopt_rms_norm_backward(dn, h0, gain, rstd, dh.view(-1, k))
    assert torch.equal(dx.view(-1, k), want[0]) and torch.equal(dgain, want[1]) and torch.equal(dres, dx)
    assert all(torch.equal(a, b) for a, b in zip(grads[None], grads[BF16]))
    for i in (0, 1, 4):
        assert torch.equal(grads[F32][i], grads[BF16][i])
    # the default's dx is off by its two roundings at most: each a half step of
    # what it rounds, the inner one times r |gain| (1 + the row mean's share)
    (exact, size), _ = _backward(dn, h0, gain, rstd, dh.view(-1, k))
    inner = (dn.abs().double() * gain.abs().double() + (h0.double() * rstd.double()[:, None]).abs() *
             (dn.double() * gain.double() * h0.double() * rstd.double()[:, None]).abs().mean(1, keepdim=True))
    bound = inner * rstd.double()[:, None] * _half(BF16) + size * (64 + 24) * 2 * U + 2.0 ** -130
    off = (grads[BF16][2].view(-1, k).double() - exact).abs()
    assert (off <= bound + (exact.abs() + bound) * _half(BF16)).all()


def test_captured_with_an_fp32_gradient():
    """Forward and backward in one graph, replayed over new inputs between eager
    calls."""
    require_gpu()
    x, gain = torch.zeros(40, 300, dtype=BF16, device="cuda"), _random(300, 1, BF16)
    w, dy = _random((200, 300), 2, BF16, 0.1), torch.zeros(40, 200, dtype=BF16, device="cuda")

    def run(x, gain, w):
        leaves = [t.detach().clone().requires_grad_() for t in (x, gain, w)]
        y, _ = F.fp8_norm_linear(*leaves, norm_grad_dtype=F32)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))
    run(x, gain, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(x, gain, w)
    for t in (1, 2, 3, 4):
        x.copy_(_random((40, 300), 10 + t, BF16))
        dy.copy_(_random((40, 200), 20 + t, BF16))
        graph.replay()
        torch.cuda.synchronize()
        want = run(x, gain, w)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), t
