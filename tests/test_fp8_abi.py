"""Refusals of the 8-bit and norm entry points without a GPU: every call here
ends in the host checks, before the HIP runtime."""
import ctypes
import os

import pytest
import torch

from bit_companded_adam_amd import flashopt as F

A, MIS = 0x10000, 0x10001      # fake device addresses, never dereferenced
B = [A + (i << 20) for i in range(12)]      # a megabyte each
OK, EINVAL, EALIGN, EWORKSPACE = F.FLASHOPT_OK, F.FLASHOPT_EINVAL, F.FLASHOPT_EALIGN, F.FLASHOPT_EWORKSPACE
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return F.lib()


def test_sizes(L):
    for rows, cols, codes, scales in ((1, 1, 128, 16), (3, 128, 384, 48), (3, 129, 768, 48), (5, 2048, 10240, 80),
                                      (5, 2049, 10880, 160), (1000, 4096, 4096000, 32000)):
        assert L.flashopt_byte_code_bytes(rows, cols) == codes
        assert L.flashopt_byte_scale_bytes(rows, cols) == scales
        assert L.flashopt_byte_linear_workspace_bytes(rows, cols) == codes + scales
        assert (F._fp8_widths(cols)[0] * rows, F._fp8_widths(cols)[1] * rows) == (codes, scales)
    for rows, cols in ((0, 5), (5, 0), (-1, 5), (BIG, 1), (1, BIG)):
        assert L.flashopt_byte_code_bytes(rows, cols) == L.flashopt_byte_scale_bytes(rows, cols) == 0
        assert L.flashopt_rms_norm_backward_workspace_bytes(rows, cols) == 0
    assert L.flashopt_byte_code_bytes(BIG - 1, BIG - 1) > 2 ** 60
    assert L.flashopt_rms_norm_backward_workspace_bytes(7, 100) >= 400


def test_quantize_refuses(L):
    def q(x=A, wide=0, rows=4, cols=40, stride=40, fmt=0, block=0, c=B[1], s=B[2], ct=None, st=None):
        return L.flashopt_byte_quantize(x, wide, rows, cols, stride, fmt, block, c, s, ct, st, None)
    assert q(rows=0, x=None) == OK and q(cols=0, x=None, c=None, s=None) == OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(wide=2), dict(wide=-1),
                dict(x=None), dict(stride=-1), dict(c=None, s=None), dict(c=None), dict(s=None), dict(ct=A),
                dict(st=A), dict(c=None, s=None, ct=A), dict(rows=BIG - 1, cols=1 << 20), dict(fmt=2), dict(fmt=-1),
                dict(block=2), dict(block=-1), dict(fmt=2, rows=0),
                # outputs that overlap
                dict(s=B[1]), dict(s=B[1] + 496), dict(ct=B[1], st=B[3]), dict(ct=B[3], st=B[2] + 16),
                dict(ct=B[3], st=B[3] + 5104)):
        assert q(**bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(x=A + 2, wide=1), dict(c=B[1] + 8), dict(s=B[2] + 4), dict(ct=B[3] + 8, st=B[4]),
                dict(ct=B[3], st=B[4] + 8)):
        assert q(**bad) == EALIGN, bad


def test_dequantize_refuses(L):
    def d(c=A, s=A, fmt=0, rows=4, cols=40, out=A, wide=0, stride=40):
        return L.flashopt_byte_dequantize(c, s, fmt, rows, cols, out, wide, stride, None)
    assert d(rows=0, out=None) == OK and d(cols=0, out=None) == OK
    for bad in (dict(rows=-1), dict(cols=BIG), dict(wide=3), dict(out=None), dict(c=None), dict(s=None),
                dict(stride=39), dict(fmt=2)):
        assert d(**bad) == EINVAL, bad
    for bad in (dict(out=MIS), dict(out=A + 2, wide=1), dict(c=A + 4), dict(s=A + 4)):
        assert d(**bad) == EALIGN, bad


def test_product_refuses(L):
    def p(a=A, sa=A, fmt=0, b=A, sb=A, m=4, n=5, k=40, out=A, wide=0, stride=5):
        return L.flashopt_byte_product(a, sa, fmt, b, sb, m, n, k, out, wide, stride, None)
    assert p(m=0, out=None) == OK and p(n=0, out=None) == OK
    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=BIG), dict(n=BIG, stride=BIG), dict(k=BIG),
                dict(k=(1 << 24) - 127), dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None),
                dict(wide=2), dict(stride=4), dict(fmt=2), dict(fmt=-1)):
        assert p(**bad) == EINVAL, bad
    for bad in (dict(a=A + 8), dict(sa=A + 4), dict(b=A + 8), dict(sb=A + 4), dict(out=MIS),
                dict(out=A + 2, wide=1)):
        assert p(**bad) == EALIGN, bad


def test_linear_refuses(L):
    need = L.flashopt_byte_linear_workspace_bytes(4, 40)

    def f(x=A, wide=0, m=4, k=40, xs=40, w=A, sw=A, n=5, out=A, ow=0, os_=5, ws=A, nbytes=need):
        return L.flashopt_byte_linear(x, wide, m, k, xs, w, sw, n, out, ow, os_, ws, nbytes, None)
    assert f(m=0, x=None, out=None) == OK and f(n=0, out=None, os_=0) == OK
    for bad in (dict(m=-1), dict(k=-1), dict(n=-1), dict(wide=2), dict(ow=2), dict(x=None), dict(w=None),
                dict(sw=None), dict(out=None), dict(xs=-1), dict(os_=4), dict(m=BIG - 1, k=1 << 20, xs=0),
                dict(k=(1 << 24) - 127, xs=1 << 24)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(w=A + 8), dict(sw=A + 4), dict(out=MIS), dict(ws=A + 8)):
        assert f(**bad) == EALIGN, bad
    assert f(ws=None) == EWORKSPACE and f(nbytes=need - 1) == EWORKSPACE


NORM = dict(x=B[0], residual=B[1], gain=B[2], h=B[3], y=B[4], codes=B[5], scales=B[6], codes_t=B[7], scales_t=B[8],
            rstd=B[9], rows=4, cols=40, x_stride=40, residual_stride=40, h_stride=40, y_stride=40, eps=1e-6, fp32=0,
            gain_fp32=0, format=0, reserved=0)


def test_norm_refuses(L):
    def f(**changed):
        return L.flashopt_rms_norm(ctypes.byref(F.flashopt_norm_args(**{**NORM, **changed})), None)
    assert L.flashopt_rms_norm(None, None) == EINVAL
    assert f(rows=0, x=None, y=None) == OK and f(cols=0, x=None) == OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(x=None), dict(gain=None),
                dict(residual=None), dict(h=None), dict(codes=None), dict(scales=None), dict(codes_t=None),
                dict(scales_t=None), dict(y=None, codes=None, scales=None, codes_t=None, scales_t=None),
                dict(rstd=None), dict(fp32=2), dict(gain_fp32=-1), dict(format=2), dict(reserved=1), dict(eps=-1.0),
                dict(eps=float("nan")), dict(eps=float("inf")), dict(x_stride=-1), dict(residual_stride=-1),
                dict(h_stride=39), dict(y_stride=39), dict(x_stride=1 << 41),
                dict(rows=BIG - 1, cols=1 << 10, x_stride=1 << 10, residual_stride=0, h_stride=1 << 10, y_stride=1 << 10),
                # what is written overlaps what is read or written
                dict(y=B[0]), dict(y=B[1]), dict(y=B[3]), dict(h=B[0] + 2), dict(h=B[1] + 80), dict(h=B[2]),
                dict(y=B[2] + 78), dict(codes=B[0]), dict(scales=B[5] + 496), dict(codes_t=B[5]), dict(rstd=B[2] + 76),
                dict(rstd=B[4] + 4), dict(scales_t=B[6]), dict(h=B[0], x_stride=41), dict(h=B[1], h_stride=41),
                dict(x=B[0], x_stride=80, y=B[0] + 78, y_stride=80),
                dict(residual=B[0], residual_stride=100, h=B[0] + 20, h_stride=200)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(residual=B[1] + 1), dict(gain=B[2] + 1), dict(h=B[3] + 1), dict(y=B[4] + 1),
                dict(x=B[0] + 2, fp32=1), dict(gain=B[2] + 2, gain_fp32=1), dict(codes=B[5] + 8),
                dict(scales=B[6] + 8), dict(codes_t=B[7] + 4), dict(scales_t=B[8] + 1), dict(rstd=B[9] + 2)):
        assert f(**bad) == EALIGN, bad


GRAD = dict(dy=B[0], dh=B[1], h=B[2], gain=B[3], rstd=B[4], dx=B[5], dgain=B[6], workspace=B[7],
            workspace_bytes=1 << 20, rows=4, cols=40, dy_stride=40, dh_stride=40, h_stride=40, dx_stride=40, fp32=0,
            gain_fp32=0)


def test_norm_backward_refuses(L):
    def f(**changed):
        return L.flashopt_rms_norm_backward(ctypes.byref(F.flashopt_norm_grad_args(**{**GRAD, **changed})), None)
    assert L.flashopt_rms_norm_backward(None, None) == EINVAL
    assert f(cols=0, dy=None) == OK and f(rows=0, dgain=None, dy=None) == OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(cols=32769), dict(dy=None),
                dict(h=None), dict(gain=None), dict(rstd=None), dict(dx=None, dgain=None), dict(fp32=2),
                dict(gain_fp32=2), dict(dy_stride=-1), dict(dh_stride=-1), dict(h_stride=-1), dict(dx_stride=39),
                dict(dx=B[2]), dict(dx=B[0] + 2), dict(dx=B[0], dx_stride=48), dict(dgain=B[3]), dict(dgain=B[5]),
                dict(workspace=B[0] - 4096), dict(dx=B[3]), dict(dx=B[4]), dict(workspace=B[6])):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(dy=MIS), dict(dh=B[1] + 1), dict(h=B[2] + 2, fp32=1), dict(gain=B[3] + 1), dict(rstd=B[4] + 2),
                dict(dx=B[5] + 1), dict(dgain=B[6] + 1), dict(workspace=B[7] + 8)):
        assert f(**bad) == EALIGN, bad
    need = L.flashopt_rms_norm_backward_workspace_bytes(4, 40)
    assert f(workspace=None) == EWORKSPACE and f(workspace_bytes=need - 1) == EWORKSPACE


def test_binding_refuses(L):
    x, gain = torch.zeros(4, 40), torch.zeros(40)
    eight = torch.zeros(1, 128).to(torch.float8_e4m3fn)
    for call in (lambda: F.flashopt_byte_quantize(x), lambda: F.FP8Weight(x),
                 lambda: F.fp8_linear(x, torch.zeros(3, 40)), lambda: F.flashopt_rms_norm(x, gain),
                 lambda: F.rms_norm(x, gain), lambda: F.fp8_norm_linear(x, gain, torch.zeros(3, 40)),
                 lambda: F.flashopt_rms_norm_backward(x, x, gain, torch.zeros(4)),
                 lambda: F.FP8Tensor(eight, torch.zeros(16, dtype=torch.uint8), 1, 40)):
        with pytest.raises(ValueError, match="device"):
            call()
    for call in (lambda: F.fp8_linear(x, torch.zeros(3, 41)), lambda: F.rms_norm(x, torch.zeros(41)),
                 lambda: F.fp8_norm_linear(x, torch.zeros(41), torch.zeros(3, 40)),
                 lambda: F.fp8_norm_linear(x, gain, torch.zeros(3, 41)), lambda: F.rms_norm(x, torch.zeros(1, 40))):
        with pytest.raises(ValueError, match="do not match"):
            call()
    for residual in (torch.zeros(4, 41), torch.zeros(4, 40).bfloat16(), torch.zeros(40)):
        with pytest.raises(ValueError, match="residual must be"):
            F.rms_norm(x, gain, residual)
    with pytest.raises(ValueError, match="matrix"):
        F.flashopt_byte_quantize(torch.zeros(4))
    for call in (lambda: F.fp8_linear(x, torch.zeros(3, 40), grad_dtype=torch.bfloat16),
                 lambda: F.FP8Tensor.empty(3, 4, "cpu", torch.int8)):
        with pytest.raises((ValueError, KeyError)):
            call()
    for codes, scales, match in ((torch.zeros(1, 128, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), "codes must be"),
                                 (eight, torch.zeros(16), "scales must be uint8")):
        with pytest.raises(ValueError, match=match):
            F.FP8Tensor(codes, scales, 1, 40)
