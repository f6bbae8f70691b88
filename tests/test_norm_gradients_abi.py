"""The type of the gradient that the norm's backward pass takes, without a GPU:
refusals of the C entry point and of fp8_norm_linear, and what fp8_norm_linear
asks the product for.  Every call ends in the host checks."""
import ctypes

import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from tests.test_fp8_abi import B, EALIGN, EINVAL, GRAD, OK, L  # noqa: F401
from tests.test_fp8_binding import calls  # noqa: F401

BF16, F32 = torch.bfloat16, torch.float32


def test_backward_refuses(L):  # noqa: F811
    def f(**changed):
        return L.flashopt_rms_norm_backward(ctypes.byref(F.flashopt_norm_grad_args(**{**GRAD, **changed})), None)
    assert f(rows=0, dgain=None, dy_fp32=1) == f(cols=0, dy_fp32=1) == OK
    for bad in (dict(dy_fp32=2), dict(dy_fp32=-1), dict(reserved=1), dict(dy_fp32=2, rows=0, dgain=None),
                # an fp32 dy is no place for a bf16 dx, and reaches twice as far
                dict(dy_fp32=1, dx=B[0]), dict(dy_fp32=1, dx=B[0], dy_stride=20), dict(dy_fp32=1, dgain=B[0] + 600),
                dict(dy_fp32=1, dx=B[2])):
        assert f(**bad) == EINVAL, bad
    assert f(dy_fp32=1, dy=B[0] + 2) == f(dy_fp32=0, fp32=1, dy=B[0] + 2) == EALIGN


def test_packed_arguments_are_the_structure():
    """The binding packs what the header's structures say, in their order."""
    for packed, structure in ((F._NORM_ARGS, F.flashopt_norm_args), (F._NORM_GRAD_ARGS, F.flashopt_norm_grad_args)):
        names = [name for name, _ in structure._fields_]
        values = [0.5 if kind is ctypes.c_double else i + 1 for i, (_, kind) in enumerate(structure._fields_)]
        got = structure.from_buffer_copy(packed.pack(*values))
        assert packed.size == ctypes.sizeof(structure) and [getattr(got, n) for n in names] == values


def test_the_type_between_product_and_norm(calls, monkeypatch):  # noqa: F811
    """x's type by default, fp32 where asked for, nothing else."""
    asked, given = [], []
    product, backward = F.flashopt_byte_product, F.flashopt_rms_norm_backward
    monkeypatch.setattr(F, "flashopt_byte_product", lambda a, b, dtype: asked.append(dtype) or product(a, b, dtype))
    monkeypatch.setattr(F, "flashopt_rms_norm_backward",
                        lambda dy, *args: given.append(dy.dtype) or backward(dy, *args))
    for dtype, choice, want in ((BF16, None, BF16), (BF16, BF16, BF16), (BF16, F32, F32), (F32, None, F32),
                                (F32, F32, F32)):
        x, gain = torch.zeros(4, 64, dtype=dtype, requires_grad=True), torch.zeros(64, requires_grad=True)
        w = torch.zeros(3, 64, dtype=BF16, requires_grad=True)
        F.fp8_norm_linear(x, gain, w, norm_grad_dtype=choice)[0].sum().backward()
        assert asked == [dtype, want, BF16] and given == [want]      # y, the norm's gradient, dw
        assert (x.grad.dtype, gain.grad.dtype, w.grad.dtype) == (dtype, F32, BF16)
        del asked[:], given[:]
    for dtype, choice in ((BF16, torch.float16), (F32, BF16), (BF16, torch.float8_e4m3fn)):
        with pytest.raises(ValueError, match="norm_grad_dtype must be"):
            F.fp8_norm_linear(torch.zeros(4, 64, dtype=dtype), gain, w, norm_grad_dtype=choice)
