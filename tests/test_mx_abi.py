"""Refusals of the MXFP4 entry points without a GPU: every call here ends in
the host checks, before the HIP runtime."""
import os

import pytest
import torch

from bit_companded_adam_amd import flashopt as F

A, MIS = 0x10000, 0x10001      # fake device addresses, never dereferenced
OK, EINVAL, EALIGN, EWORKSPACE = F.FLASHOPT_OK, F.FLASHOPT_EINVAL, F.FLASHOPT_EALIGN, F.FLASHOPT_EWORKSPACE
BIG = 1 << 31


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return F.lib()


def test_sizes(L):
    for rows, cols, codes in ((1, 1, 64), (3, 128, 192), (3, 129, 384), (1000, 4096, 2048000)):
        assert L.flashopt_mx_code_bytes(rows, cols) == codes
        assert L.flashopt_mx_scale_bytes(rows, cols) == codes // 16
    for rows, cols in ((0, 5), (5, 0), (-1, 5), (BIG, 1), (1, BIG)):
        assert L.flashopt_mx_code_bytes(rows, cols) == L.flashopt_mx_scale_bytes(rows, cols) == 0
    assert L.flashopt_mx_code_bytes(BIG - 1, BIG - 1) > 2 ** 60
    assert L.flashopt_mx_linear_workspace_bytes(3, 129) == 384 + 32
    assert L.flashopt_mx_linear_workspace_bytes(0, 129) == 0


def test_quantize_refuses(L):
    def q(x=A, wide=0, rows=4, cols=40, stride=40, c=A, s=A, ct=None, st=None):
        return L.flashopt_mx_quantize(x, wide, rows, cols, stride, c, s, ct, st, None)
    assert q(rows=0, x=None) == OK and q(cols=0, x=None, c=None, s=None) == OK
    for bad in (dict(rows=-1), dict(cols=-1), dict(rows=BIG), dict(cols=BIG), dict(wide=2), dict(wide=-1),
                dict(x=None), dict(stride=-1), dict(c=None, s=None), dict(c=None), dict(s=None), dict(ct=A),
                dict(st=A), dict(c=None, s=None, ct=A), dict(rows=BIG - 1, cols=1 << 20)):
        assert q(**bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(x=A + 2, wide=1), dict(c=A + 8), dict(s=A + 2), dict(ct=A + 8, st=A),
                dict(ct=A, st=A + 1)):
        assert q(**bad) == EALIGN, bad


def test_dequantize_refuses(L):
    def d(c=A, s=A, rows=4, cols=40, out=A, wide=0, stride=40):
        return L.flashopt_mx_dequantize(c, s, rows, cols, out, wide, stride, None)
    assert d(rows=0, out=None) == OK and d(cols=0, out=None) == OK
    for bad in (dict(rows=-1), dict(cols=BIG), dict(wide=3), dict(out=None), dict(c=None), dict(s=None),
                dict(stride=39)):
        assert d(**bad) == EINVAL, bad
    for bad in (dict(out=MIS), dict(out=A + 2, wide=1), dict(c=A + 4), dict(s=A + 1)):
        assert d(**bad) == EALIGN, bad


def test_product_refuses(L):
    def p(a=A, sa=A, b=A, sb=A, m=4, n=5, k=40, out=A, wide=0, stride=5):
        return L.flashopt_mx_product(a, sa, b, sb, m, n, k, out, wide, stride, None)
    assert p(m=0, out=None) == OK and p(n=0, out=None) == OK
    for bad in (dict(m=-1), dict(n=-1), dict(k=-1), dict(m=BIG), dict(n=BIG, stride=BIG), dict(k=BIG), dict(k=(1 << 25) - 127),
                dict(a=None), dict(sa=None), dict(b=None), dict(sb=None), dict(out=None), dict(wide=2),
                dict(stride=4)):
        assert p(**bad) == EINVAL, bad
    for bad in (dict(a=A + 8), dict(sa=A + 2), dict(b=A + 8), dict(sb=A + 2), dict(out=MIS),
                dict(out=A + 2, wide=1)):
        assert p(**bad) == EALIGN, bad


def test_linear_refuses(L):
    need = L.flashopt_mx_linear_workspace_bytes(4, 40)

    def f(x=A, wide=0, m=4, k=40, xs=40, w=A, sw=A, n=5, out=A, ow=0, os_=5, ws=A, nbytes=need):
        return L.flashopt_mx_linear(x, wide, m, k, xs, w, sw, n, out, ow, os_, ws, nbytes, None)
    assert f(m=0, x=None, out=None) == OK and f(n=0, out=None, os_=0) == OK
    for bad in (dict(m=-1), dict(k=-1), dict(n=-1), dict(wide=2), dict(ow=2), dict(x=None), dict(w=None),
                dict(sw=None), dict(out=None), dict(xs=-1), dict(os_=4), dict(m=BIG - 1, k=1 << 20, xs=0)):
        assert f(**bad) == EINVAL, bad
    for bad in (dict(x=MIS), dict(w=A + 8), dict(sw=A + 1), dict(out=MIS), dict(ws=A + 8)):
        assert f(**bad) == EALIGN, bad
    assert f(ws=None) == EWORKSPACE and f(nbytes=need - 1) == EWORKSPACE


def test_binding_refuses(L):
    x = torch.zeros(4, 40)
    for call in (lambda: F.flashopt_mx_quantize(x), lambda: F.MXWeight(x),
                 lambda: F.mx_linear(x, torch.zeros(3, 40)),
                 lambda: F.MXTensor(torch.zeros(64, dtype=torch.uint8), torch.zeros(4, dtype=torch.uint8), 1, 40)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="do not match"):
        F.mx_linear(x, torch.zeros(3, 41))
    with pytest.raises(ValueError, match="matrix"):
        F.flashopt_mx_quantize(torch.zeros(4))
