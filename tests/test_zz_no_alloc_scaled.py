"""The allocation-free list step with a grad_scale: every stored byte equal to
the workspace list step's with the same scale, over two steps, for variants of
the storage; and without one again afterwards."""
import ctypes

import numpy as np
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import host, require_gpu

pytestmark = pytest.mark.gpu

SIZES = [1 << 14, 3000, 70001, 1, 33, 4096]


@pytest.mark.parametrize("mb,comp,qs,layout", [(24, True, True, "blocked"), (32, False, True, "streams"),
                                               (None, True, False, "streams")])
def test_scaled_noalloc_step(mb, comp, qs, layout):
    require_gpu()
    L = F.lib()
    ref, got = [[F.TensorState(W.init_param(n, device="cuda", seed=300 + i), mb, qs, state_layout=layout)
                 for i, n in enumerate(SIZES)] for _ in range(2)]
    ws = torch.empty(F.flashopt_adamw_workspace_bytes(len(SIZES)), dtype=torch.uint8, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    for t, factor in ((1, 0.3), (2, 5.0), (3, None)):
        scale = None if factor is None else torch.tensor([factor], device="cuda")
        grads = [W.make_grad(n, t, device="cuda", stream_id=i) for i, n in enumerate(SIZES)]
        args = F.make_args(t, master_bits=mb, companded=comp, quantize_states=qs, state_layout=layout,
                           grad_scale=scale, **W.HP_DEFAULT)
        F.flashopt_adamw_step(F.descriptor_array(ref, grads), args, ws)
        status = L.flashopt_adamw_step_noalloc(F.descriptor_array(got, grads), len(SIZES), ctypes.byref(args),
                                               stream)
        assert status == F.FLASHOPT_OK, F.status_str(status)
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            for x, y in ((a.param, b.param), (a.rho, b.rho), (a.m_codes, b.m_codes), (a.m_scales, b.m_scales),
                         (a.v_codes, b.v_codes), (a.v_scales, b.v_scales)):
                if x is not None:
                    assert (host(x.view(torch.uint8)).view(np.uint8) == host(y.view(torch.uint8)).view(np.uint8)).all(), t
