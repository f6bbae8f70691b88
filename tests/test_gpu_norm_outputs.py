"""Outputs of flashopt_rms_norm together, by the C entry point: y beside codes
along rows, along columns and both; and rows with infinities and NaN on the way
to every one of them."""
import ctypes

import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import COLS, _random

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2


def _same(a, b):
    return torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scales, b.scales)


def _call(x, gain, residual, eps, with_y, with_rows, with_cols, kind):
    """(y, h, rows, cols, rstd) of one call, each filled with 77 before."""
    rows, cols = x.shape
    y, h = torch.full_like(x, 77), torch.full_like(x, 77)
    rstd = torch.full((rows,), 77.0, device="cuda")
    q, t = F.FP8Tensor.empty(rows, cols, "cuda", kind), F.FP8Tensor.empty(cols, rows, "cuda", kind)
    q._buffer.fill_(77), t._buffer.fill_(77)
    args = F.flashopt_norm_args(
        x=x.data_ptr(), residual=None if residual is None else residual.data_ptr(), gain=gain.data_ptr(),
        h=None if residual is None else h.data_ptr(), y=y.data_ptr() if with_y else None,
        codes=q.code_ptr if with_rows else None, scales=q.scale_ptr if with_rows else None,
        codes_t=t.code_ptr if with_cols else None, scales_t=t.scale_ptr if with_cols else None, rstd=rstd.data_ptr(),
        rows=rows, cols=cols, x_stride=cols, residual_stride=cols, h_stride=cols, y_stride=cols, eps=eps,
        fp32=int(x.dtype == F32), gain_fp32=int(gain.dtype == F32), format=F.FORMATS[kind], reserved=0)
    assert F.lib().flashopt_rms_norm(ctypes.byref(args), F._stream(None)) == F.FLASHOPT_OK
    return y, h, q, t, rstd


@pytest.mark.parametrize("cols", [c for c in COLS if c not in (8, 127, 513, 1032, 16384)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_values_and_codes_in_one_call(cols, dtype):
    require_gpu()
    for rows, kind in ((1, E4M3), (130, E4M3), (33, E5M2)):
        x, gain = _random((rows, cols), cols + rows, dtype), _random(cols, cols, BF16 if cols % 2 else dtype)
        for residual in (None, _random((rows, cols), cols + rows + 1, dtype, 3.0)):
            r0 = torch.empty(rows, device="cuda")
            y0, h0 = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, rstd=r0)
            (q0, t0), _ = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, output="both", dtype=kind)
            for with_rows, with_cols in ((True, False), (False, True), (True, True)):
                y, h, q, t, rstd = _call(x, gain, residual, 1e-5, True, with_rows, with_cols, kind)
                assert torch.equal(y, y0) and torch.equal(rstd, r0)
                assert torch.equal(h, h0) if residual is not None else (h == 77).all()
                assert _same(q, q0) if with_rows else (q._buffer == 77).all()
                assert _same(t, t0) if with_cols else (t._buffer == 77).all()
                again = _call(x, gain, residual, 1e-5, False, with_rows, with_cols, kind)
                assert (again[0] == 77).all() and (not with_rows or _same(again[2], q0)) and (
                    not with_cols or _same(again[3], t0))


@pytest.mark.parametrize("cols", [5, 100, 700, 2500, 33000])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_rows_that_are_not_finite(cols, dtype, kind):
    """Along rows such a row's groups are NaN; along columns, a group that a NaN
    falls into, for each of its rows; all others as if the row were another.
    Every output is that of the codec on the fp32 y."""
    require_gpu()
    for rows in (5, 300):
        x = _random((rows, cols), 1, dtype)
        for row, at, bad in ((1, min(cols - 1, 3), "inf"), (2, cols - 1, "-inf"), (rows - 1, cols // 2, "nan")):
            x[row, at] = float(bad)
        gain = _random(cols, 2, F32)
        for residual in (None, _random((rows, cols), 3, dtype)):
            y, h, q, t, rstd = _call(x, gain, residual, 1e-6, True, True, True, kind)
            h = x if residual is None else h
            y32 = (h.float() * rstd[:, None]) * gain
            assert torch.equal(y.isnan(), y32.isnan()) and torch.equal(y.nan_to_num(9.0), y32.to(dtype).nan_to_num(9.0))
            # an infinity: r is 0, it is NaN, and the rest of its row zeros; a NaN: the whole row
            nan = torch.zeros(rows, cols, dtype=torch.bool, device="cuda")
            nan[1, min(cols - 1, 3)], nan[2, cols - 1], nan[rows - 1] = True, True, True
            assert torch.equal(y32.isnan(), nan) and (y32[1:3][~nan[1:3]] == 0).all()
            want, want_t = F.flashopt_byte_quantize(y32, "both", dtype=kind)
            assert _same(q, want) and _same(t, want_t)
            for layout, mine in (("rows", q), ("cols", t)):
                alone, _ = F.flashopt_rms_norm(x, gain, residual, output=layout, dtype=kind)
                assert _same(alone, mine)
            groups = F.flashopt_byte_dequantize(t).isnan()
            pad = torch.zeros(-(-rows // 128) * 128, cols, dtype=torch.bool, device="cuda")
            pad[:rows] = nan
            some = pad.view(-1, 128, cols).any(1).repeat_interleave(128, 0)[:rows]
            assert torch.equal(groups, some.t())
