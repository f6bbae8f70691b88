"""Outputs of a quantization that share memory, refused without a GPU: every
call here ends in the host checks, before the HIP runtime."""
import os

import pytest

from bit_companded_adam_amd import flashopt as F

X, A = 0x100000, 0x10000       # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return F.lib()


def test_quantize_refuses_outputs_that_overlap(L):
    """A 128 x 128 matrix: 8192 bytes of codes and 512 of scales each way.
    (Neighbours in one buffer are what MXTensor.empty makes.)"""
    def q(c, s, ct, st):
        return L.flashopt_mx_quantize(X, 0, 128, 128, 128, c, s, ct, st, None)
    code, scale = L.flashopt_mx_code_bytes(128, 128), L.flashopt_mx_scale_bytes(128, 128)
    assert (code, scale) == (8192, 512)
    a, b, c = A + code, A + code + scale, A + 2 * code + scale
    for bad in ((A, a, A, a), (A, a, A, c), (A, a, b, a), (A, a - 4, None, None), (None, None, A, A + 64),
                (A, c, A + code - 16, c + code), (A + 256, A, b, c), (A, c, b + code, c + scale - 4)):
        assert q(*bad) == F.FLASHOPT_EINVAL, bad
