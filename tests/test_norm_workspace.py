"""Bytes of the norm's backward workspace, without a GPU: one partial row of
dgain for each workgroup there is, and a buffer made for the largest pass serves
all smaller ones."""
import ctypes

import pytest

from bit_companded_adam_amd import flashopt as F
from tests.test_fp8_abi import EINVAL, EWORKSPACE, GRAD, B, L  # noqa: F401

COLS = [1, 40, 511, 512, 513, 1023, 1024, 1025, 2047, 2048, 2049, 2304, 4096, 4097, 8192, 16384, 20000, 32768]
ROWS = [1, 2, 3, 4, 5, 255, 256, 257, 511, 512, 513, 1024, 2047, 2048, 2049, 8192, 1 << 20, (1 << 31) - 1]


def _groups(rows, cols):
    """Workgroups of the launch: four rows to one up to 1024 columns, two to a CU
    up to 2048, one beyond."""
    return min(-(-rows // 4), 512) if cols <= 1024 else min(rows, 512 if cols <= 2048 else 256)


def test_sizes(L):  # noqa: F811
    f = L.flashopt_rms_norm_backward_workspace_bytes
    assert f(1, 32768) == 4 * 32768 and f(8192, 4096) == 4 * 256 * 4096 and f(8192, 2048) == 4 * 512 * 2048
    for rows in ROWS:
        for cols in COLS:
            own = 4 * cols * _groups(rows, cols)
            widest = max(4 * c * _groups(rows, c) for c in {*COLS, cols} if c <= cols)
            assert f(rows, cols) == max(own, widest), (rows, cols)
            assert f(rows, cols) <= 4 * 512 * cols


def test_never_falls(L):  # noqa: F811
    f = L.flashopt_rms_norm_backward_workspace_bytes
    sizes = [[f(r, c) for c in COLS] for r in ROWS]
    for row in sizes:
        assert row == sorted(row)
    for column in zip(*sizes):
        assert list(column) == sorted(column)


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 20000), (3, 1500), (7, 1000), (300, 4096)])
def test_what_is_needed_is_what_is_asked_for(L, rows, cols):  # noqa: F811
    need = L.flashopt_rms_norm_backward_workspace_bytes(rows, cols)
    big = {n: B[0] + (i << 32) for i, n in enumerate(("dy", "dh", "h", "gain", "rstd", "dx", "dgain", "workspace"))}

    def f(**changed):
        sizes = dict(rows=rows, cols=cols, dy_stride=cols, dh_stride=cols, h_stride=cols, dx_stride=cols)
        args = F.flashopt_norm_grad_args(**{**GRAD, **big, **sizes, **changed})
        return L.flashopt_rms_norm_backward(ctypes.byref(args), None)
    assert f(workspace_bytes=need - 1) == EWORKSPACE
    # enough, and refused for another reason: dgain lies on its last byte
    assert f(workspace_bytes=need, dgain=big["workspace"] + (need - 4) // 4 * 4) == EINVAL


def test_a_workspace_over_what_is_read_is_refused_whatever_the_rows(L):  # noqa: F811
    """Inputs that lie behind the bytes that few rows take, inside those that
    many do and that the caller has handed over."""
    def f(**changed):
        return L.flashopt_rms_norm_backward(ctypes.byref(F.flashopt_norm_grad_args(**{**GRAD, **changed})), None)
    for rows in (1, 4, 4096):
        assert f(rows=rows, workspace=B[0] - 4096) == EINVAL
    need = L.flashopt_rms_norm_backward_workspace_bytes(4, 40)
    assert need <= 4096
    assert f(workspace=B[0] - 160, workspace_bytes=need, dx=B[0] - 160 + need - 2) == EINVAL
