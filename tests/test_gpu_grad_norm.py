"""The gradient norm, clipping in place and the clipped steps on the GPU.

The norm is checked against a 64-bit sum: its squares and sums are fp64, so
only the last rounding to fp32 counts (half a unit, 2^-24).  Clipped gradients
and clipped steps are compared bit for bit, with the scale the GPU returned."""
import math
import threading

import numpy as np
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import host, require_gpu, u16

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
HALF = 2.0 ** -24 * (1 + 2.0 ** -20)      # one fp32 rounding, over the fp64 error of any list here


def _grads(sizes, seed=0, scale=1e-3):
    """Every third gradient fp32, the others bf16."""
    return [W.make_grad(n, 1, device="cuda", seed=seed, scale=scale, stream_id=i,
                        dtype=F32 if i % 3 == 2 else BF16) for i, n in enumerate(sizes)]


def _norm64(grads):
    parts = [float((g.double() ** 2).sum()) for g in grads]
    return math.sqrt(math.fsum(parts))


def _check(out, grads64_norm, max_norm):
    norm, scale = out.double().tolist()
    # below 2^-126 fp32 values lie 2^-149 apart: the rounding is off by at
    # most half of that, 2^-150, whatever the value (the norm of 5000 times
    # 1e-44 is 6.9e-43, 495 such steps)
    assert abs(norm - grads64_norm) <= max(HALF * grads64_norm, 2.0 ** -150)
    want = min(1.0, max_norm / (grads64_norm + 1e-6))
    assert abs(scale - want) <= HALF * want


SIZES = {
    "one": [1],
    "odd": [1, 7, 31, 33, 4095, 4096, 4097, 12289],
    "empty-among": [0, 5, 0, 0, 8193, 0],
    "mid": [65536 + 3, 1 << 20, 17],
    "table": [64 * i + 1 for i in range(65)],          # over 64 tensors: the staged table
    "large": [(1 << 24) + 5, 4096 * 300, 100003],
}


@pytest.mark.parametrize("name", SIZES)
def test_norm_and_clip(name):
    require_gpu()
    grads = _grads(SIZES[name])
    norm = _norm64(grads)
    for max_norm in (0.3 * norm, 2.0 * norm + 1.0, float("inf"), 0.0):
        print(f"{name}: max_norm {max_norm}", flush=True)
        _check(F.flashopt_grad_norm(grads, max_norm), norm, max_norm)
    before = [g.clone() for g in grads]
    out = F.flashopt_grad_clip(grads, 2.0 * norm + 1.0)            # nothing to clip
    assert float(out[1]) == 1.0
    for g, b in zip(grads, before):
        assert torch.equal(g, b)
    again = F.flashopt_grad_norm(grads, 1.0)
    assert torch.equal(again, F.flashopt_grad_norm(grads, 1.0))     # the same bits each time
    out = F.flashopt_grad_clip(grads, 0.3 * norm)
    _check(out, norm, 0.3 * norm)
    for g, b in zip(grads, before):
        assert torch.equal(g, (b.float() * out[1]).to(b.dtype))


@pytest.mark.parametrize("n", [8, 70], ids=["args", "table"])
def test_unaligned_views(n):
    """Gradients at any element of a flat buffer, neighbours untouched."""
    require_gpu()
    sizes = [1 + 997 * i % 9001 for i in range(n)]
    for dtype in (BF16, F32):
        flat = W.make_grad(sum(sizes) + 2 * n, 1, device="cuda", dtype=dtype)
        views, gaps, at = [], [], 0
        for s in sizes:
            gaps.append(flat[at:at + 2])
            views.append(flat[at + 1:at + 1 + s])
            at += s + 2
        before = flat.clone()
        norm = _norm64(views)
        _check(F.flashopt_grad_norm(views, norm), norm, norm)
        out = F.flashopt_grad_clip(views, norm / 3)
        want, at = before.clone(), 0
        for s in sizes:
            part = want[at + 1:at + 1 + s]
            part.copy_((part.float() * out[1]).to(dtype))
            at += s + 2
        assert torch.equal(flat, want)


def test_extremes_and_non_finite():
    """Squares beyond fp32's range both ways; infinities and NaN."""
    require_gpu()
    for dtype, value in ((F32, 1e30), (F32, 1e-30), (BF16, 2.0 ** 100), (BF16, 2.0 ** -100), (F32, 1e-44)):
        g = [torch.full((5000,), value, dtype=dtype, device="cuda")]
        _check(F.flashopt_grad_norm(g, 1.0), _norm64(g), 1.0)
    for bad, norm, scale in ((float("inf"), float("inf"), 0.0), (float("nan"), float("nan"), float("nan"))):
        g = _grads([10000, 3])
        g[0][9999] = bad
        out = F.flashopt_grad_norm(g, 1.0).tolist()
        assert str(out[0]) == str(norm) and str(out[1]) == str(scale)
    out = F.flashopt_grad_norm([torch.full((9,), float("inf"), device="cuda")]).tolist()
    assert out[0] == float("inf") and math.isnan(out[1])
    zero = [torch.zeros(77, device="cuda")]
    assert F.flashopt_grad_norm(zero, 1e-3).tolist() == [0.0, 1.0]
    assert F.flashopt_grad_norm([], 1.0).tolist() == [0.0, 1.0]
    assert F.flashopt_grad_clip([torch.zeros(0, device="cuda")], 0.0).tolist() == [0.0, 0.0]


def test_norm_counts_a_repeated_gradient_twice():
    require_gpu()
    g = _grads([1000])[0]
    _check(F.flashopt_grad_norm([g, g], 1.0), math.sqrt(2) * _norm64([g]), 1.0)
    with pytest.raises(F.FlashoptError, match="EINVAL"):
        F.flashopt_grad_clip([g, g[10:20]], 1.0)
    plan = F.GradPlan([g, g])
    _check(plan.norm(1.0), math.sqrt(2) * _norm64([g]), 1.0)
    with pytest.raises(F.FlashoptError, match="EINVAL"):
        plan.clip(1.0)


@pytest.mark.parametrize("n", [5, 100], ids=["short", "long"])
def test_plan_and_other_stream(n):
    require_gpu()
    grads = _grads([1 + 517 * i for i in range(n)])
    norm = _norm64(grads)
    plan = F.GradPlan(grads)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [plan.norm(0.5 * norm), F.flashopt_grad_norm(grads, 0.5 * norm)]
    torch.cuda.synchronize()
    outs += [plan.norm(0.5 * norm, stream=side), F.flashopt_grad_norm(grads, 0.5 * norm, stream=side),
             F.flashopt_grad_norm(grads, 0.5 * norm, stream=side.cuda_stream)]
    side.synchronize()
    for out in outs:
        _check(out, norm, 0.5 * norm)
        assert torch.equal(out, outs[0])
    before = [g.clone() for g in grads]
    out = plan.clip(0.5 * norm)
    for g, b in zip(grads, before):
        assert torch.equal(g, (b.float() * out[1]).to(b.dtype))


@pytest.mark.parametrize("n", [5, 100], ids=["call", "plan"])
def test_captured_norm_and_clipped_step(n):
    """Norm and clipped step in one graph: replays with new gradients, eager
    work between them, equal eager steps on a second optimizer."""
    require_gpu()
    sizes = [33 + 1021 * i for i in range(n)]
    params = [W.init_param(s, device="cuda", seed=i) for i, s in enumerate(sizes)]
    a = F.FlashAdamW([p.clone() for p in params], **W.HP_DEFAULT)
    b = F.FlashAdamW([p.clone() for p in params], **W.HP_DEFAULT)
    bufs = [torch.zeros(s, dtype=BF16, device="cuda") for s in sizes]
    out = torch.zeros(2, device="cuda")
    norms = F.GradPlan(bufs)
    plan = a.plan(bufs, step=1, grad_scale=out[1:])
    norm = (lambda: F.flashopt_grad_norm(bufs, 0.01, out=out)) if n <= 64 else (lambda: norms.norm(0.01, out=out))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm()
        plan.launch()
    for t in (1, 2, 3, 4):
        grads = [W.make_grad(s, t, device="cuda", stream_id=i) for i, s in enumerate(sizes)]
        for d, g in zip(bufs, grads):
            d.copy_(g)
        plan.set_step(t)
        graph.replay()
        eager = b.step(grads, max_norm=0.01)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), t
        assert float(out[1]) < 1.0
        for x, y in zip(a.states, b.states):
            assert (u16(x.param) == u16(y.param)).all()
            assert torch.equal(x.block, y.block)


def test_capture_of_a_long_list_is_refused():
    """Its table is staged from the host, which a graph cannot hold."""
    require_gpu()
    grads = [torch.ones(8, device="cuda") for _ in range(65)]
    out = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for call in (F.flashopt_grad_norm, F.flashopt_grad_clip):
            with pytest.raises(ValueError, match="GradPlan"):
                call(grads, 1.0, out=out)
        F.flashopt_grad_norm(grads[:64], 1.0, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        # 512 ones: the norm is one rounding of an fp64 square root
        assert out[0].item() == float(torch.tensor(512.0).sqrt())


def test_threads_on_streams_of_their_own():
    """Norms from several host threads at once, each on its own stream."""
    require_gpu()
    lists = [[W.make_grad(50_000 + 1000 * i, k, device="cuda", stream_id=i) for i in range(n)]
             for k, n in enumerate((3, 40, 90, 130))]
    want = [F.flashopt_grad_norm(l, 0.5) for l in lists]
    torch.cuda.synchronize()
    got, errors = [[] for _ in lists], []

    def work(k):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                got[k].append(F.flashopt_grad_norm(lists[k], 0.5, stream=stream))
            stream.synchronize()
        except Exception as e:                     # raised again below
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(len(lists))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for k, outs in enumerate(got):
        assert len(outs) == 20 and all(torch.equal(o, want[k]) for o in outs)


# ------------------------------------------------------------ clipped steps

def _oracle_scaled_step(orc, p, st, g32, t, hp, mb, comp, qs):
    """One step from the oracle's parts on an fp32 gradient."""
    h = orc.hparams(step=t, master_bits=mb, companded=comp, quantize_states=qs,
                    fp32_param=p.dtype == np.float32, **hp)
    ms = orc.MOMENTUM if comp else orc.MOMENTUM_LINEAR
    vs = orc.VARIANCE if comp else orc.VARIANCE_LINEAR
    m, v = (orc.dequantize(*st["m"], ms), orc.dequantize(*st["v"], vs)) if qs else (st["m"], st["v"])
    if p.dtype == np.float32:
        theta = p
    elif mb:
        theta = orc.reconstruct(p, st["rho"], mb)
    else:
        theta = (p.astype(np.uint32) << 16).view(np.float32)
    theta, m, v = orc.adamw_update(theta, m, v, g32, h)
    st["m"], st["v"] = (orc.quantize(m, ms), orc.quantize(v, vs)) if qs else (m, v)
    if p.dtype == np.float32:
        return theta
    if mb:
        p, st["rho"] = orc.split(theta, mb)
        return p
    return u16(torch.from_numpy(theta).to(BF16))


VARIANTS = [(24, True, True, "blocked", BF16), (24, True, True, "streams", BF16),
            (32, True, True, "blocked", BF16), (24, False, True, "streams", BF16),
            (None, True, True, "blocked", BF16), (24, True, False, None, BF16),
            (None, True, False, None, BF16), (None, True, True, "blocked", F32),
            (None, True, False, None, F32)]


@pytest.mark.parametrize("mb,comp,qs,layout,dtype", VARIANTS)
@pytest.mark.parametrize("how", ["list", "tensor"])
def test_scaled_adamw_equals_the_oracle(orc, mb, comp, qs, layout, dtype, how):
    require_gpu()
    sizes = [1, 31, 1024, 5000 + 17]
    params = [W.init_param(n, device="cuda", seed=20 + i, dtype=dtype) for i, n in enumerate(sizes)]
    opt = F.FlashAdamW(params, master_bits=mb, companded=comp, quantize_states=qs, state_layout=layout,
                       **W.HP_DEFAULT)
    bits = (lambda x: host(x)) if dtype == F32 else u16
    hosts = [bits(p) for p in params]
    sts = []
    for n in sizes:
        z = np.zeros(n, np.float32)
        st = {"m": z, "v": z}
        if qs:
            st = {"m": orc.quantize(z, orc.MOMENTUM), "v": orc.quantize(z, orc.VARIANCE)}
        if mb:
            st["rho"] = np.zeros(n, orc.rho_dtype(mb))
        sts.append(st)
    for t, factor in ((1, 0.37), (2, 1.0), (3, 3.0e-3)):
        scale = torch.tensor([factor], device="cuda")
        grads = [W.make_grad(n, t, device="cuda", stream_id=i, dtype=dtype) for i, n in enumerate(sizes)]
        if how == "list":
            opt.step(grads, grad_scale=scale)
        else:
            for i, g in enumerate(grads):
                opt.step_tensor(i, g, grad_scale=scale)
        for i, g in enumerate(grads):
            g32 = host(g.float()) * np.float32(factor)
            hosts[i] = _oracle_scaled_step(orc, hosts[i], sts[i], g32, t, W.HP_DEFAULT, mb, comp, qs)
            s, st = opt.states[i], sts[i]
            assert (bits(s.param) == hosts[i]).all(), (t, i)
            if mb:
                assert (host(s.rho) == st["rho"]).all()
            if qs:
                assert (host(s.m_codes) == st["m"][0]).all() and (u16(s.m_scales) == st["m"][1]).all()
                assert (host(s.v_codes) == st["v"][0]).all() and (u16(s.v_scales) == st["v"][1]).all()
            else:
                assert (host(s.m_codes) == st["m"]).all() and (host(s.v_codes) == st["v"]).all()


@pytest.mark.parametrize("mb,comp,qs,layout", [(24, True, True, "streams"), (32, False, True, "blocked"),
                                               (None, True, False, None)])
@pytest.mark.parametrize("how", ["list", "tensor", "plan"])
def test_scaled_sgd_equals_the_oracle(orc, mb, comp, qs, layout, how):
    require_gpu()
    sizes = [1, 33, 4096 + 5]
    params = [W.init_param(n, device="cuda", seed=40 + i) for i, n in enumerate(sizes)]
    opt = F.FlashSGD(params, master_bits=mb, companded=comp, quantize_states=qs, state_layout=layout,
                     **W.SGD_DEFAULT)
    spec = orc.MOMENTUM if comp else orc.MOMENTUM_LINEAR
    thetas = [host(p.float()) for p in params]
    bufs = [np.zeros(n, np.float32) for n in sizes]
    for t, factor in ((1, 0.41), (2, 7.0)):
        scale = torch.tensor([factor], device="cuda")
        grads = [W.make_grad(n, t, device="cuda", stream_id=i) for i, n in enumerate(sizes)]
        if how == "list":
            opt.step(grads, grad_scale=scale)
        elif how == "tensor":
            for i, g in enumerate(grads):
                opt.step_tensor(i, g, grad_scale=scale)
        else:
            opt.plan(grads, step=t, grad_scale=scale).launch()
        h = orc.sgd_hparams(step=t, master_bits=mb, companded=comp, quantize_states=qs, **W.SGD_DEFAULT)
        for i, g in enumerate(grads):
            theta, buf = orc.sgd_update(thetas[i], bufs[i], host(g.float()) * np.float32(factor), h)
            s = opt.states[i]
            if qs:
                codes, scales = orc.quantize(buf, spec)
                assert (host(s.m_codes) == codes).all() and (u16(s.m_scales) == scales).all()
                buf = orc.dequantize(codes, scales, spec)
            else:
                assert (host(s.m_codes) == buf).all()
            if mb:
                bits, rho = orc.split(theta, mb)
                assert (host(s.rho) == rho).all()
                theta = orc.reconstruct(bits, rho, mb)
            else:
                bits = u16(torch.from_numpy(theta).to(BF16))
                theta = (bits.astype(np.uint32) << 16).view(np.float32)
            assert (u16(s.param) == bits).all(), (t, i)
            thetas[i], bufs[i] = theta, buf


def test_max_norm_step():
    """step(max_norm=) is the norm followed by the scaled step; a NaN
    gradient reaches every parameter, as it does a clipped eager step."""
    require_gpu()
    sizes = [5000, 17, 70000]
    make = lambda: F.FlashAdamW([W.init_param(n, device="cuda", seed=i) for i, n in enumerate(sizes)],
                                **W.HP_DEFAULT)
    a, b = make(), make()
    for t in (1, 2):
        grads = [W.make_grad(n, t, device="cuda", stream_id=i) for i, n in enumerate(sizes)]
        out = a.step(grads, max_norm=0.05)
        ref = F.flashopt_grad_norm(grads, 0.05)
        assert torch.equal(out, ref) and float(out[1]) < 1
        assert b.step(grads, grad_scale=ref[1:]) is None
        for x, y in zip(a.states, b.states):
            assert torch.equal(x.param, y.param) and torch.equal(x.block, y.block)
    with pytest.raises(ValueError, match="exclude"):
        a.step(grads, max_norm=1.0, grad_scale=ref[1:])
    with pytest.raises(ValueError, match="grad_scale"):
        a.step(grads, grad_scale=torch.ones(1))
    assert a.t == 2
    grads[1][3] = float("nan")
    a.step(grads, max_norm=1.0)
    assert all(torch.isnan(s.param).all() for s in a.states)
