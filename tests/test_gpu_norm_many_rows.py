"""The gain's gradient over many rows, against 64 bits.

The launch has 512 workgroups up to 2048 columns and 256 beyond, and no more
than there are rows for (up to 1024 columns a workgroup takes four at once).  A
thread adds its rows' terms in fp32, one after another, four such sums are added
where four rows go at once, and the workgroups' are added in 64 bits.  Each
addition is off by at most 2^-24 of the sum of magnitudes so far, and each term
h r by 2^-24 of itself."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests._gpu import require_gpu
from tests.test_gpu_norm import U, _half, _random

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def additions(rows, cols):
    at_once = 4 if cols <= 1024 else 1
    groups = min(-(-rows // at_once), 512 if cols <= 2048 else 256)
    return -(-rows // (groups * at_once)) + at_once - 1


@pytest.mark.parametrize("rows,cols,dtype", [(200000, 64, BF16), (200001, 77, F32), (60000, 1500, BF16),
                                             (60000, 2304, BF16), (30001, 2049, F32), (20000, 8200, BF16),
                                             (3000, 20000, F32), (5000, 4096, BF16), (2049, 1024, F32), (1, 300, F32)])
def test_dgain(rows, cols, dtype):
    require_gpu()
    h, dy = _random((rows, cols), 1, dtype, 2.0), _random((rows, cols), 2, dtype)
    gain, rstd = _random(cols, 3, F32), torch.empty(rows, device="cuda")
    F.flashopt_rms_norm(h, gain, rstd=rstd)
    for into in (F32, BF16):
        _, dgain = F.flashopt_rms_norm_backward(dy, h, gain.to(into), rstd, need_dx=False)
        want = torch.zeros(cols, dtype=torch.float64, device="cuda")
        size = want.clone()
        for at in range(0, rows, 4096):
            terms = dy[at:at + 4096].double() * (h[at:at + 4096].double() * rstd[at:at + 4096, None].double())
            want += terms.sum(0)
            size += terms.abs().sum(0)
        bound = size * (additions(rows, cols) + 1) * U * 1.001 + 2.0 ** -140
        bound = bound + (want.abs() + bound) * U                    # the sum in 64 bits, rounded to fp32
        assert dgain.dtype == into
        assert ((dgain.double() - want).abs() <= bound + (want.abs() + bound) * (_half(into) if into == BF16 else 0)).all()
        again = F.flashopt_rms_norm_backward(dy, h, gain.to(into), rstd, need_dx=False)[1]
        assert torch.equal(again, dgain)
