"""Refusals of the gradient norm, clipping and grad_scale arguments without a
GPU: every call here ends in the host checks, before the HIP runtime."""
import ctypes
import os

import pytest
import torch

from bit_companded_adam_amd import flashopt as F

A16, A4, MIS = 0x10000, 0x10004, 0x10001      # fake device addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(F._LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return F.lib()


def _list(*grads):
    return (F.flashopt_grad * max(1, len(grads)))(*[F.flashopt_grad(*g) for g in grads]), len(grads)


@pytest.mark.parametrize("name", ["flashopt_grad_norm", "flashopt_grad_clip"])
def test_list_calls_refuse(L, name):
    def call(*grads, max_norm=1.0, out=A16, ws=A16, nbytes=1 << 20, n=None):
        arr, count = _list(*grads)
        return getattr(L, name)(arr if grads else None, count if n is None else n, max_norm, out, ws,
                                nbytes, None)
    ok = (A16, 1000, 0)
    need = L.flashopt_grad_workspace_bytes(1)
    assert call(ok, nbytes=need - 1) == F.FLASHOPT_EWORKSPACE
    assert call(ok, ws=None) == F.FLASHOPT_EWORKSPACE
    assert call(ok, ws=A16 + 8, nbytes=need) == F.FLASHOPT_EALIGN
    assert call(n=-1) == F.FLASHOPT_EINVAL
    assert call(n=1) == F.FLASHOPT_EINVAL                                  # NULL list
    assert call((A16, -1, 0)) == F.FLASHOPT_EINVAL
    assert call((None, 5, 0)) == F.FLASHOPT_EINVAL
    assert call((A16, 5, 2)) == F.FLASHOPT_EINVAL
    assert call((MIS, 5, 0)) == F.FLASHOPT_EALIGN
    assert call((A16 + 2, 5, 1)) == F.FLASHOPT_EALIGN                      # fp32 at 2 bytes
    assert call((A16 + 2, 5, 0), ws=None) == F.FLASHOPT_EWORKSPACE         # bf16 there is fine
    assert call((A16, 1 << 44, 0)) == F.FLASHOPT_EINVAL                    # over 2^31 - 1 chunks
    assert call((A16, (1 << 63) - 1, 0)) == F.FLASHOPT_EINVAL
    for bad in (-1.0, float("nan")):
        assert call(ok, max_norm=bad) == F.FLASHOPT_EINVAL
    assert call(ok, max_norm=float("inf"), ws=None) == F.FLASHOPT_EWORKSPACE
    assert call(ok, out=None) == F.FLASHOPT_EINVAL
    assert call(ok, out=A16 + 2) == F.FLASHOPT_EALIGN
    assert call(ok, out=A4, ws=None) == F.FLASHOPT_EWORKSPACE


def test_clip_refuses_overlapping_gradients(L):
    def clip(*grads, ws=None):
        arr, n = _list(*grads)
        return L.flashopt_grad_clip(arr, n, 1.0, A16, ws, 1 << 20, None)
    assert clip((A16, 100, 0), (A16, 100, 0), ws=A16) == F.FLASHOPT_EINVAL
    assert clip((A16 + 198, 10, 0), (A16, 100, 0), ws=A16) == F.FLASHOPT_EINVAL
    assert clip((A16, 50, 1), (A16 + 100, 4, 0), ws=A16) == F.FLASHOPT_EINVAL
    assert clip((A16 + 200, 10, 0), (A16, 100, 0)) == F.FLASHOPT_EWORKSPACE     # neighbours are fine
    assert clip((A16, 100, 0), (A16, 0, 0)) == F.FLASHOPT_EWORKSPACE            # an empty one too
    # a norm may count a gradient twice
    arr, n = _list((A16, 100, 0), (A16, 100, 0))
    assert L.flashopt_grad_norm(arr, n, 1.0, A16, None, 0, None) == F.FLASHOPT_EWORKSPACE


def test_workspace_sizes(L):
    assert L.flashopt_grad_workspace_bytes(0) == 0 and L.flashopt_grad_plan_bytes(0) == 0
    assert L.flashopt_grad_workspace_bytes(1) == L.flashopt_grad_workspace_bytes(64)
    assert L.flashopt_grad_workspace_bytes(65) >= L.flashopt_grad_workspace_bytes(64) + 65 * 24
    assert L.flashopt_grad_plan_bytes(1) >= L.flashopt_grad_workspace_bytes(1) + 24
    assert F.flashopt_grad_workspace_bytes(290) == F.flashopt_grad_plan_bytes(290)


def test_plan_refuses(L):
    info = F.flashopt_grad_plan_info()

    def plan(*grads, buf=A16, nbytes=1 << 20, inf=info, n=None):
        arr, count = _list(*grads)
        return L.flashopt_grad_plan(arr if grads else None, count if n is None else n, buf, nbytes,
                                    ctypes.byref(inf) if inf is not None else None, None)
    ok = (A16, 5000, 0)
    need = L.flashopt_grad_plan_bytes(1)
    assert plan(ok, inf=None) == F.FLASHOPT_EINVAL
    assert plan(ok, buf=None) == F.FLASHOPT_EWORKSPACE
    assert plan(ok, nbytes=need - 1) == F.FLASHOPT_EWORKSPACE
    assert plan(ok, buf=A16 + 8, nbytes=need) == F.FLASHOPT_EALIGN
    assert plan((A16, -1, 0)) == F.FLASHOPT_EINVAL
    assert plan((MIS, 1, 0)) == F.FLASHOPT_EALIGN
    assert plan(n=-1) == F.FLASHOPT_EINVAL
    assert plan() == F.FLASHOPT_OK and (info.n_tensors, info.total_chunks) == (0, 0)
    for call in (L.flashopt_grad_plan_norm, L.flashopt_grad_plan_clip):
        def launch(fields=(1, 2, 0), buf=A16, max_norm=1.0, out=A16):
            return call(ctypes.byref(F.flashopt_grad_plan_info(*fields)), buf, max_norm, out, None)
        assert call(None, A16, 1.0, A16, None) == F.FLASHOPT_EINVAL
        assert launch((-1, 2, 0)) == F.FLASHOPT_EINVAL
        assert launch((1, -2, 0)) == F.FLASHOPT_EINVAL
        assert launch((0, 2, 0)) == F.FLASHOPT_EINVAL
        assert launch(buf=None) == F.FLASHOPT_EWORKSPACE
        assert launch(buf=A16 + 8) == F.FLASHOPT_EALIGN
        assert launch(max_norm=-1.0) == F.FLASHOPT_EINVAL
        assert launch(max_norm=float("nan")) == F.FLASHOPT_EINVAL
        assert launch(out=None) == F.FLASHOPT_EINVAL
        assert launch(out=A16 + 1) == F.FLASHOPT_EALIGN
    assert L.flashopt_grad_plan_clip(ctypes.byref(F.flashopt_grad_plan_info(2, 2, 1)), A16, 1.0, A16,
                                     None) == F.FLASHOPT_EINVAL


def test_grad_scale_arguments(L):
    """grad_scale: 4-byte aligned; a plan's launches and set_step agree on
    whether there is one."""
    t = (F.flashopt_tensor * 1)(F.flashopt_tensor(A16, A16, A16, A16, A16, A16, A16, 4096))
    a, s = F.make_args(1), F.make_sgd_args(1)
    assert a.grad_scale is None and s.grad_scale is None
    a.grad_scale, s.grad_scale = A16 + 2, A16 + 2
    assert L.flashopt_adamw_step(t, 1, ctypes.byref(a), A16, 1 << 20, None) == F.FLASHOPT_EALIGN
    assert L.flashopt_sgd_step(t, 1, ctypes.byref(s), A16, 1 << 20, None) == F.FLASHOPT_EALIGN
    assert L.flashopt_adamw_step_tensor(t, ctypes.byref(a), None) == F.FLASHOPT_EALIGN
    a.grad_scale, s.grad_scale = A4, A4
    assert L.flashopt_adamw_step(t, 1, ctypes.byref(a), None, 0, None) == F.FLASHOPT_EWORKSPACE
    assert L.flashopt_sgd_step(t, 1, ctypes.byref(s), None, 0, None) == F.FLASHOPT_EWORKSPACE
    plain, scaled = F.flashopt_adamw_plan_info(1, 4, 24, 1), F.flashopt_adamw_plan_info(1, 4, 24, 1, 0, 0, 0, 1)
    for info, args, want in ((plain, a, F.FLASHOPT_EINVAL), (scaled, a, F.FLASHOPT_EWORKSPACE),
                             (scaled, F.make_args(1), F.FLASHOPT_EINVAL)):
        assert L.flashopt_adamw_plan_set_step(ctypes.byref(info), ctypes.byref(args), None, None) == want
    bad = F.flashopt_adamw_plan_info(1, 4, 24, 1, 0, 0, 0, 2)
    assert L.flashopt_adamw_plan_launch(ctypes.byref(bad), A16, None) == F.FLASHOPT_EINVAL
    sp, ss = F.flashopt_sgd_plan_info(1, 4, 24, 1), F.flashopt_sgd_plan_info(1, 4, 24, 1, 0, 0, 1)
    for info, args, want in ((sp, s, F.FLASHOPT_EINVAL), (ss, s, F.FLASHOPT_EWORKSPACE),
                             (ss, F.make_sgd_args(1), F.FLASHOPT_EINVAL)):
        assert L.flashopt_sgd_plan_set_step(ctypes.byref(info), ctypes.byref(args), None, None) == want
    bad = F.flashopt_sgd_plan_info(1, 4, 24, 1, 0, 0, 2)
    assert L.flashopt_sgd_plan_launch(ctypes.byref(bad), A16, None) == F.FLASHOPT_EINVAL


def test_binding_refuses(L):
    for call in (lambda g: F.flashopt_grad_norm([g]), lambda g: F.flashopt_grad_clip([g], 1.0),
                 lambda g: F.GradPlan([g])):
        with pytest.raises(ValueError, match="device"):
            call(torch.zeros(8))
        with pytest.raises(ValueError, match="bf16 or fp32"):
            call(torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError, match="grad_scale"):
        F.make_args(1, grad_scale=torch.ones(1))                # a host tensor
