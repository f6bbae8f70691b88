"""The root-mean-square norm, its 8-bit outputs and its gradients on the GPU,
and the layer that joins it to the 8-bit product.

Forward: the sum is compared bit for bit (one fp32 addition, rounded), r within
one rounding of the 64-bit value, and y within the roundings that follow it:
r's, two products' and the output's own.  8-bit outputs are compared byte for
byte with the codec's on the fp32 y that r gives.  Backward: against the formula
in 64 bits, with a bound for each fp32 operation."""
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
U = 2.0 ** -24                       # half a step of fp32


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _random(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _forward(x, gain, residual, eps):
    """(h, r, y) by the formula: h in its own type, r and y in 64 bits."""
    h = x if residual is None else (x.float() + residual.float()).to(x.dtype)
    r = 1.0 / (h.double().square().mean(1) + eps).sqrt()
    return h, r, h.double() * r[:, None] * gain.double()


def _check_values(y, rstd, want_r, want_y, dtype):
    assert ((rstd.double() - want_r).abs() <= want_r * U * 1.001).all()
    assert y.dtype == dtype
    # r, then two products in fp32 (values below fp32's normal range: half a
    # step of the smallest), then the output's rounding
    bound = want_y.abs() * (3.01 * U) + 2.0 ** -149
    if dtype == BF16:
        bound = bound + (want_y.abs() + bound) * _half(BF16) + 2.0 ** -134
    assert ((y.double() - want_y).abs() <= bound).all()


COLS = [1, 7, 8, 9, 127, 128, 129, 500, 512, 513, 1001, 1024, 1032, 2048, 2049, 4096, 5000, 8192, 8200, 16384, 16391,
        32768, 32776, 40001]


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("with_residual", [False, True])
def test_forward(cols, dtype, with_residual):
    require_gpu()
    for rows in (1, 3, 33, 130):
        x = _random((rows, cols), cols + rows, dtype)
        residual = _random((rows, cols), cols + rows + 1, dtype, 3.0) if with_residual else None
        gain_type = BF16 if cols % 2 else dtype
        gain = _random(cols, cols, gain_type)
        h, r, y = _forward(x, gain, residual, 1e-5)
        rstd = torch.full((rows,), 7.0, device="cuda")
        got, got_h = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, rstd=rstd)
        assert torch.equal(got_h, h) and (with_residual or got_h is x)
        _check_values(got, rstd, r, y, dtype)
        # 8 bits: of the same fp32 products, r being what the kernel says it is
        y32 = (h.float() * rstd[:, None]) * gain.float()
        for kind in (E4M3, E5M2) if rows == 33 else (E4M3,):
            rows8, h8 = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, output="rows", dtype=kind)
            (both, cols8), _ = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, output="both", dtype=kind)
            alone, _ = F.flashopt_rms_norm(x, gain, residual, eps=1e-5, output="cols", dtype=kind)
            want, want_t = F.flashopt_byte_quantize(y32, "both", dtype=kind)
            assert torch.equal(h8, h)
            for a, b in ((rows8, want), (both, want), (cols8, want_t), (alone, want_t)):
                assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
                assert torch.equal(a.scales, b.scales)


def test_forward_is_the_same_in_any_company():
    """A row's result does not depend on the rows around it."""
    require_gpu()
    for cols in (300, 2048, 9000):
        x, gain, res = _random((700, cols), 1, BF16), _random(cols, 2, BF16), _random((700, cols), 3, BF16)
        y, h = F.flashopt_rms_norm(x, gain, res)
        for i in (0, 5, 699):
            one, one_h = F.flashopt_rms_norm(x[i:i + 1], gain, res[i:i + 1])
            assert torch.equal(one, y[i:i + 1]) and torch.equal(one_h, h[i:i + 1])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_views_and_the_sum_in_place(dtype):
    """Row strides and odd offsets; h into a view, into residual or x itself;
    what lies around stays as it was."""
    require_gpu()
    for cols in (40, 301, 2050, 33000):
        base, other = _random((70, cols + 9), 1, dtype), _random((70, cols + 5), 2, dtype)
        gain = _random(cols, 3, F32)
        for a, b in ((base[:, 1:cols + 1], other[:, 3:cols + 3]), (base[::3, 8:cols + 8], other[::3, :cols]),
                     (base[5:6, 2:cols + 2].expand(20, cols), other[:20, 1:cols + 1])):
            h, r, y = _forward(a, gain, b, 1e-6)
            wide = torch.full((a.shape[0] + 1, 2 * cols + 6), 77.0, dtype=dtype, device="cuda")
            out, hv = wide[1:, 1:cols + 1], wide[1:, cols + 3:2 * cols + 3]
            rstd = torch.empty(a.shape[0], device="cuda")
            got, got_h = F.flashopt_rms_norm(a, gain, b, out=out, h=hv, rstd=rstd)
            assert got is out and got_h is hv and torch.equal(hv, h)
            _check_values(out, rstd, r, y, dtype)
            want = out.clone()
            out.fill_(77), hv.fill_(77)
            assert (wide == 77).all()
            for which in (0, 1):
                mine = [base.clone(), other.clone()]
                if a.stride(0) == 0 and which == 0:
                    continue                            # rows that are one cannot each take a sum
                views = [torch.as_strided(m, t.shape, t.stride(), t.storage_offset()) for m, t in zip(mine, (a, b))]
                got, got_h = F.flashopt_rms_norm(views[0], gain, views[1], h=views[which])
                assert torch.equal(got_h, h) and torch.equal(got, want)
                q, _ = F.flashopt_rms_norm(a, gain, b, output="both")
                mine = [base.clone(), other.clone()]
                views = [torch.as_strided(m, t.shape, t.stride(), t.storage_offset()) for m, t in zip(mine, (a, b))]
                q2, got_h = F.flashopt_rms_norm(views[0], gain, views[1], h=views[which], output="both")
                assert torch.equal(got_h, h)
                for s, t in zip(q, q2):
                    assert torch.equal(s._buffer, t._buffer)


def test_extreme_rows():
    """Rows of zeros, of the largest and smallest values: the sum of squares
    stays in range.  Rows with infinities and NaN as the formula says."""
    require_gpu()
    for cols in (100, 2500, 33000):
        x = _random((8, cols), 1, F32)
        x[0] = 0
        x[1] *= 1e30
        x[2] *= 1e-30
        x[3, 3] = float("inf")
        x[4, 4] = float("nan")
        x[5] = 3e38
        x[6] = 2.0 ** -149
        gain = torch.ones(cols, device="cuda")
        y, _ = F.flashopt_rms_norm(x, gain, eps=0.0)
        assert torch.isnan(y[0]).all()                       # 0 / 0
        assert torch.isnan(y[3, 3]) and (y[3, :3] == 0).all() and (y[3, 4:] == 0).all()
        assert torch.isnan(y[4]).all()
        ok = [1, 2, 5, 6, 7]
        _, r, want = _forward(x[ok], gain, None, 0.0)
        inside = (r < 3e38)                                  # row 6's r is above fp32's range
        assert ((y[ok][inside].double() - want[inside]).abs() <= want[inside].abs() * 3.01 * U).all()
        y, _ = F.flashopt_rms_norm(x, gain, eps=1e-6)
        assert (y[0] == 0).all() and (y[6].abs() < 1e-40).all()
        q, _ = F.flashopt_rms_norm(x, gain, eps=1e-6, output="rows")
        v = F.flashopt_byte_dequantize(q)
        assert torch.isnan(v[3, :min(cols, 128)]).all() and torch.isnan(v[4]).all()
        assert torch.isfinite(v[[0, 1, 2, 5, 6, 7]]).all() and (v[0] == 0).all()


def test_empty():
    require_gpu()
    gain = torch.ones(40, device="cuda")
    x = torch.zeros(0, 40, device="cuda")
    y, h = F.flashopt_rms_norm(x, gain, x.clone())
    assert y.shape == h.shape == (0, 40)
    q, _ = F.flashopt_rms_norm(x, gain, output="both")
    assert q[0].rows == 0 and q[1].cols == 0
    dx, dgain = F.flashopt_rms_norm_backward(x, x, gain, torch.zeros(0, device="cuda"))
    assert dx.shape == (0, 40) and torch.equal(dgain, torch.zeros(40, device="cuda"))
    z = torch.zeros(3, 0, device="cuda")
    y, _ = F.flashopt_rms_norm(z, torch.zeros(0, device="cuda"))
    assert y.shape == (3, 0)


# -------------------------------------------------------------- backward

def _backward(dy, h, gain, rstd, dh):
    """((dx, its magnitude), (dgain, its magnitude)) in 64 bits; r as given."""
    dy, h, gain, r = dy.double(), h.double(), gain.double(), rstd.double()[:, None]
    u, t = dy * gain, h * r
    c, c_size = (u * t).mean(1, keepdim=True), (u * t).abs().mean(1, keepdim=True)
    e = 0.0 if dh is None else dh.double()
    dx = r * (u - t * c) + e
    size = r * (u.abs() + t.abs() * c_size) + (0.0 if dh is None else e.abs())
    return (dx, size), ((dy * t).sum(0), (dy * t).abs().sum(0))


def _check_backward(dx, dgain, dy, h, gain, rstd, dh):
    rows, cols = h.shape
    (want_x, size_x), (want_g, size_g) = _backward(dy, h, gain, rstd, dh)
    # c: each term three roundings, then at most cols additions (in fact a tree
    # of eight a lane); its use and the rest of dx seven more
    if dx is not None:
        bound = size_x * (min(cols, 64) + 24) * 2 * U + 2.0 ** -140
        assert ((dx.double() - want_x).abs() <= bound + (want_x.abs() + bound) * (_half(BF16) if dx.dtype == BF16 else U)).all()
    # dgain: each term two roundings, then at most ceil(rows / 512) + 4 fp32
    # additions before the 64-bit sum
    if dgain is not None:
        bound = size_g * (rows / 512 + 12) * U + 2.0 ** -140
        assert ((dgain.double() - want_g).abs() <= bound + (want_g.abs() + bound) * _half(dgain.dtype)).all()


@pytest.mark.parametrize("cols", [c for c in COLS if c <= 32768])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_backward(cols, dtype):
    require_gpu()
    for rows in (1, 3, 33, 130):
        h, dy = _random((rows, cols), cols + rows, dtype, 2.0), _random((rows, cols), cols + rows + 1, dtype, 1e-3)
        dh = _random((rows, cols), cols + rows + 2, dtype, 1e-3) if rows != 3 else None
        gain = _random(cols, cols, dtype if cols % 2 else F32)
        rstd = torch.empty(rows, device="cuda")
        F.flashopt_rms_norm(h, gain, rstd=rstd)
        dx, dgain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh)
        _check_backward(dx, dgain, dy, h, gain, rstd, dh)
        only_x, none = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh, need_dgain=False)
        assert none is None and torch.equal(only_x, dx)
        none, only_gain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh, need_dx=False)
        assert none is None and torch.equal(only_gain, dgain)
        for place in (dy, dh):
            if place is not None:
                mine = place.clone()
                into, _ = F.flashopt_rms_norm_backward(mine if place is dy else dy, h, gain, rstd,
                                                       mine if place is dh else dh, dx=mine)
                assert into is mine and torch.equal(mine, dx)


@pytest.mark.parametrize("rows", [511, 512, 513, 2047, 2048, 2049, 5000])
def test_backward_many_rows(rows):
    require_gpu()
    for cols, dtype in ((64, F32), (777, BF16), (1500, F32), (4096, BF16)):
        h, dy = _random((rows, cols), rows, dtype, 2.0), _random((rows, cols), rows + 1, dtype)
        gain, rstd = _random(cols, 3, F32), torch.empty(rows, device="cuda")
        F.flashopt_rms_norm(h, gain, rstd=rstd)
        dx, dgain = F.flashopt_rms_norm_backward(dy, h, gain, rstd)
        _check_backward(dx, dgain, dy, h, gain, rstd, None)
        again = F.flashopt_rms_norm_backward(dy, h, gain, rstd)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dgain)


def test_backward_views():
    require_gpu()
    for dtype in (BF16, F32):
        for cols in (41, 1300, 5001):
            base = _random((70, 4 * cols + 9), 1, dtype)
            parts = [base[:, 1 + i * (cols + 1):1 + i * (cols + 1) + cols] for i in range(3)]
            gain, rstd = _random(cols, 2, BF16), torch.empty(70, device="cuda")
            F.flashopt_rms_norm(parts[1], gain, rstd=rstd)
            want, want_gain = F.flashopt_rms_norm_backward(*[p.contiguous() for p in parts[:2]], gain, rstd,
                                                           parts[2].contiguous())
            wide = torch.full((71, cols + 5), 77.0, dtype=dtype, device="cuda")
            dx, dgain = F.flashopt_rms_norm_backward(parts[0], parts[1], gain, rstd, parts[2], dx=wide[1:, 3:cols + 3])
            assert torch.equal(dx, want) and torch.equal(dgain, want_gain)
            wide[1:, 3:cols + 3] = 77
            assert (wide == 77).all()


def test_gradients_against_differences():
    """The 64-bit loss moves along a direction as the kernel's gradients say:
    central differences of the formula at a step of 1e-5, whose own error is
    some 1e-9, against dx and dgain, which hold 2^-24 of their terms' sizes."""
    require_gpu()
    rows, cols = 9, 203
    x, res, gain = _random((rows, cols), 1, F32), _random((rows, cols), 2, F32), _random(cols, 3, F32)
    dy, dh = _random((rows, cols), 4, F32), _random((rows, cols), 5, F32)
    for t in (x, res, gain):
        t.requires_grad_()
    y, h = F.rms_norm(x, gain, res, eps=1e-5)
    grads = torch.autograd.grad((y, h), (x, res, gain), (dy, dh))
    assert torch.equal(grads[0], grads[1])

    def loss(x, res, gain):
        h = x + res
        r = 1.0 / (h.square().mean(1, keepdim=True) + 1e-5).sqrt()
        return float((h * r * gain * dy.double() + h * dh.double()).sum())
    # the sum as it is held: an fp32 one, so h is the point of the differences
    at = [h.detach().double(), torch.zeros(rows, cols, dtype=F64, device="cuda"), gain.detach().double()]
    for i, grad in enumerate(grads):
        d = _random(grad.shape, 7 + i, F64)
        moved = [[a + (s * d if j == i else 0) for j, a in enumerate(at)] for s in (1e-5, -1e-5)]
        slope = (loss(*moved[0]) - loss(*moved[1])) / 2e-5
        size = float((grad.double().abs() * d.abs()).sum())
        assert abs(float((grad.double() * d).sum()) - slope) <= size * 1e-5


# -------------------------------------------------------------- autograd

@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("shape,dtype", [((2, 5, 130), BF16), ((40, 700), F32)])
def test_rms_norm_gradients(with_residual, shape, dtype):
    """Every set of gradients that may be asked for, and outputs that the loss
    does not use."""
    require_gpu()
    cols = shape[-1]
    x, gain, res = _random(shape, 1, dtype), _random(cols, 2, BF16), _random(shape, 3, dtype)
    dy, dh = _random(shape, 4, dtype), _random(shape, 5, dtype)
    rstd = torch.empty(x.numel() // cols, device="cuda")
    flat = [t.view(-1, cols) for t in (x, res, dy, dh)]
    y0, h0 = F.flashopt_rms_norm(flat[0], gain, flat[1] if with_residual else None, rstd=rstd)
    for use_y, use_h in ((True, True), (True, False), (False, True)):
        if not with_residual and use_h:
            continue
        for need in range(1, 8):
            leaves = [t.clone().requires_grad_(bool(need >> i & 1)) for i, t in enumerate((x, gain, res))]
            if not with_residual and not (leaves[0].requires_grad or leaves[1].requires_grad):
                continue
            y, h = F.rms_norm(leaves[0], leaves[1], leaves[2] if with_residual else None)
            assert torch.equal(y, y0.view(shape)) and torch.equal(h, h0.view(shape)) and y.shape == h.shape == shape
            outs = [(o, g) for o, g, use in ((y, dy, use_y), (h, dh, use_h)) if use and o.requires_grad]
            torch.autograd.backward([o for o, _ in outs], [g for _, g in outs])
            if use_y:
                dx, dgain = F.flashopt_rms_norm_backward(flat[2], h0, gain, rstd, flat[3] if use_h else None)
            else:
                dx, dgain = flat[3], None
            for leaf, want in zip(leaves, (dx, dgain, dx if with_residual else None)):
                if leaf.requires_grad and want is not None:
                    assert torch.equal(leaf.grad, want.view(leaf.shape)), (use_y, use_h, need)
                else:
                    assert leaf.grad is None


def test_rms_norm_saves_what_changes_are_seen_in():
    """The gain or h changed in place between the passes: the backward refuses."""
    require_gpu()
    x, res = _random((4, 64), 1, BF16).requires_grad_(), _random((4, 64), 2, BF16)
    gain = torch.nn.Parameter(_random(64, 3, BF16))
    y, h = F.rms_norm(x, gain, res)
    with torch.no_grad():
        gain.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y, h = F.rms_norm(x, gain, res)
    with torch.no_grad():
        h.mul_(2)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
@pytest.mark.parametrize("shape,n,dtype", [((1, 40), 30, BF16), ((2, 50, 300), 129, BF16), ((200, 260), 1100, F32)])
def test_norm_linear(with_residual, held, kind, shape, n, dtype):
    """The layer is its parts: the same bits as the library's calls one by one,
    for every set of gradients and outputs."""
    require_gpu()
    k = shape[-1]
    x, gain, res = _random(shape, 1, dtype), _random(k, 2, dtype), _random(shape, 3, dtype)
    w = _random((n, k), 4, dtype, 0.1)
    dy, dh = _random((*shape[:-1], n), 5, dtype, 1e-3), _random(shape, 6, dtype, 1e-3)
    flat, rflat = x.view(-1, k), res.view(-1, k) if with_residual else None
    rstd = torch.empty(flat.shape[0], device="cuda")
    (rows, cols), h0 = F.flashopt_rms_norm(flat, gain, rflat, output="both", rstd=rstd)
    w_rows, w_cols = F.flashopt_byte_quantize(w, "both", block=True)
    y0 = F.flashopt_byte_product(rows, w_rows, dtype)
    dy_rows, dy_cols = F.flashopt_byte_quantize(dy.view(-1, n), "both", dtype=kind)
    dn = F.flashopt_byte_product(dy_rows, w_cols, dtype)
    dw = F.flashopt_byte_product(dy_cols, cols, dtype)
    for use_h in (False, True) if with_residual else (False,):
        dx, dgain = F.flashopt_rms_norm_backward(dn, h0, gain, rstd, dh.view(-1, k) if use_h else None)
        for need in range(1, 16):
            leaves = [t.clone().requires_grad_(bool(need >> i & 1)) for i, t in enumerate((x, gain, w, res))]
            if not with_residual and not need & 7:
                continue
            weight = F.FP8Weight(leaves[2]) if held else leaves[2]
            y, h = F.fp8_norm_linear(leaves[0], leaves[1], weight, leaves[3] if with_residual else None,
                                     grad_dtype=kind)
            assert torch.equal(y, y0.view(y.shape)) and torch.equal(h, h0.view(shape)) and y.shape == dy.shape
            outs = [(y, dy)] + ([(h, dh)] if use_h and h.requires_grad else [])
            torch.autograd.backward([o for o, _ in outs], [g for _, g in outs])
            for leaf, want in zip(leaves, (dx, dgain, dw, dx if with_residual else None)):
                if leaf.requires_grad and want is not None:
                    assert torch.equal(leaf.grad, want.view(leaf.shape)), (use_h, need)
                else:
                    assert leaf.grad is None


def test_norm_linear_only_the_sum_used():
    require_gpu()
    x, res = _random((6, 64), 1, BF16).requires_grad_(), _random((6, 64), 2, BF16).requires_grad_()
    gain, w = _random(64, 3, BF16).requires_grad_(), _random((32, 64), 4, BF16).requires_grad_()
    dh = _random((6, 64), 5, BF16)
    _, h = F.fp8_norm_linear(x, gain, w, res)
    h.backward(dh)
    assert torch.equal(x.grad, dh) and torch.equal(res.grad, dh) and gain.grad is None and w.grad is None


def test_norm_linear_without_gradients():
    require_gpu()
    x, gain, w = _random((6, 64), 1, BF16), _random(64, 3, BF16).requires_grad_(), _random((32, 64), 4, BF16)
    want, _ = F.fp8_norm_linear(x, gain, w)
    with torch.no_grad():
        y, h = F.fp8_norm_linear(x, gain, w.requires_grad_(), x.clone())
        assert not y.requires_grad and not h.requires_grad
        y, h = F.fp8_norm_linear(x, gain, w)
        assert torch.equal(y, want) and h is x


# -------------------------------------------------- together, as in a model

def test_serving_path():
    """A decode step's path through two layers: the residual's addition and the
    norm to 8 bits, the product; each kept tensor is what the parts give, on
    a stream of its own too."""
    require_gpu()
    for m in (1, 3, 40, 300):
        x, res = _random((m, 512), 1, BF16), _random((m, 512), 2, BF16)
        gains = [_random(512, 3 + i, BF16) for i in range(2)]
        weights = [F.flashopt_byte_quantize(_random((512, 512), 5 + i, BF16, 0.05), block=True) for i in range(2)]

        def layers(stream=None):
            h, y = res, x
            for gain, w in zip(gains, weights):
                q, h = F.flashopt_rms_norm(y, gain, h, output="rows", stream=stream)
                y = F.flashopt_byte_product(q, w, stream=stream)
            return y, h
        y, h = layers()
        want_y, want_h = x, res
        for gain, w in zip(gains, weights):
            n, want_h = F.flashopt_rms_norm(want_y.float(), gain, want_h.float())
            want_h = want_h.to(BF16)
            n, _ = F.flashopt_rms_norm(want_h.float(), gain)
            want_y = F.flashopt_byte_product(F.flashopt_byte_quantize(n), w)
        assert torch.equal(y, want_y) and torch.equal(h, want_h)
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        y2, h2 = layers(side)
        side.synchronize()
        assert torch.equal(y2, y) and torch.equal(h2, h)


def _model(seed=0):
    """Two layers that share a residual stream: their parameters and optimizer."""
    params = [W.init_param(96 * 64, device="cuda", seed=seed + i).view(96, 64) for i in range(2)]
    params += [W.init_param(64 * 96, device="cuda", seed=seed + 5 + i).view(64, 96) for i in range(2)]
    params += [torch.ones(64, dtype=BF16, device="cuda") for _ in range(2)]
    params = [p.clone().requires_grad_() for p in params]
    opt = F.FlashAdamW([p.detach() for p in params], **W.HP_DEFAULT)
    return params, opt, [F.FP8Weight(p) for p in params[:4]]


def _losses(params, weights, x, dy):
    """A forward and backward pass: (output, gradients)."""
    h, y = None, x
    for i in range(2):
        u, h = F.fp8_norm_linear(y, params[4 + i], weights[i], h)
        y = F.fp8_linear(torch.relu(u), weights[2 + i])
    out = y + h
    return out, torch.autograd.grad(out, params, dy)


def test_training_steps():
    """Norms, 8-bit layers, the clipped step on compressed states and new copies
    of the weights, for three steps; a second run agrees bit for bit, and each
    step moves every parameter."""
    require_gpu()

    def run():
        params, opt, weights = _model()
        seen = []
        for t in (1, 2, 3):
            out, grads = _losses(params, weights, _random((48, 64), t, BF16), _random((48, 64), 40 + t, BF16, 1e-2))
            before = [s.block.clone() for s in opt.states]
            clip = opt.step(list(grads), max_norm=0.01)
            assert float(clip[1]) < 1.0
            for w in weights:
                w.refresh()
            assert all(not torch.equal(s.block, b) for s, b in zip(opt.states, before))
            seen += [out.detach(), *grads, clip, *[p.detach().clone() for p in params]]
        return seen
    for a, b in zip(run(), run()):
        assert torch.isfinite(a).all() and torch.equal(a, b)


def test_captured_training_step():
    """The same step in one graph: replays with new inputs, eager steps of a
    second model between them, equal bits.  The captured parameters are in no
    eager graph."""
    require_gpu()
    pa, a, wa = _model()
    pb, b, wb = _model()
    x, dy = torch.zeros(48, 64, dtype=BF16, device="cuda"), torch.zeros(48, 64, dtype=BF16, device="cuda")
    grads, out = [torch.zeros_like(p) for p in pa], torch.zeros(2, device="cuda")
    norm, plan = F.GradPlan(grads), a.plan(grads, step=1, grad_scale=out[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, got = _losses(pa, wa, x, dy)
        y = y.detach()
        for g, h in zip(grads, got):
            g.copy_(h)
        norm.norm(0.01, out=out)
        plan.launch()
        for w in wa:
            w.refresh()
    for t in (1, 2, 3, 4):
        x.copy_(_random((48, 64), t, BF16))
        dy.copy_(_random((48, 64), 40 + t, BF16, 1e-2))
        plan.set_step(t)
        graph.replay()
        z, eager = _losses(pb, wb, x, dy)
        clip = b.step(list(eager), max_norm=0.01)
        for w in wb:
            w.refresh()
        torch.cuda.synchronize()
        assert torch.equal(y, z) and torch.equal(out, clip), t
        for p, q in zip([*pa, *grads], [*pb, *eager]):
            assert torch.equal(p, q), t


def test_other_stream_and_threads():
    """Calls from two host threads, each on a stream of its own."""
    require_gpu()
    import threading
    x, gain = _random((300, 1000), 1, BF16), _random(1000, 2, BF16)
    dy = _random((300, 1000), 3, BF16)
    rstd = torch.empty(300, device="cuda")
    want, _ = F.flashopt_rms_norm(x, gain, rstd=rstd)
    want_dx, want_dgain = F.flashopt_rms_norm_backward(dy, x, gain, rstd)
    torch.cuda.synchronize()
    wrong = []

    def work():
        side = torch.cuda.Stream()
        for _ in range(20):
            r = torch.empty(300, device="cuda")
            y, _ = F.flashopt_rms_norm(x, gain, rstd=r, stream=side)
            dx, dgain = F.flashopt_rms_norm_backward(dy, x, gain, r, stream=side)
            side.synchronize()
            if not (torch.equal(y, want) and torch.equal(dx, want_dx) and torch.equal(dgain, want_dgain)):
                wrong.append(1)
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_offsets_past_32_bits():
    """More than 2^32 elements: the last rows are those of the last rows alone."""
    require_gpu()
    rows, cols, last = 140000, 32768, 40
    x = torch.ones(rows, cols, dtype=BF16, device="cuda")
    x[-last:] = _random((last, cols), 1, BF16)
    gain = _random(cols, 2, BF16)
    rstd, tail = torch.empty(rows, device="cuda"), torch.empty(last, device="cuda")
    q, _ = F.flashopt_rms_norm(x, gain, output="rows", rstd=rstd)
    end, _ = F.flashopt_rms_norm(x[-last:], gain, output="rows", rstd=tail)
    assert torch.equal(rstd[-last:], tail) and torch.equal(q.scales[-last:], end.scales)
    assert torch.equal(q.codes[-last:].view(torch.uint8), end.codes.view(torch.uint8))
    del q
    y, h = F.flashopt_rms_norm(x, gain, x)
    ye, he = F.flashopt_rms_norm(x[-last:], gain, x[-last:])
    assert torch.equal(y[-last:], ye) and torch.equal(h[-last:], he)
    dx, _ = F.flashopt_rms_norm_backward(y, x, gain, rstd, need_dgain=False)
    de, _ = F.flashopt_rms_norm_backward(ye, x[-last:], gain, tail, need_dgain=False)
    assert torch.equal(dx[-last:], de)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("cols", [40, 512, 1001, 4096, 8192, 16384, 20000, 32768])
def test_backward_in_place(cols, dtype):
    """dx over dy, over dh, and one gradient that is both; more rows than
    workgroups take at once, so that the next row is loaded under this one."""
    require_gpu()
    h, gain = _random((1100, cols), 1, dtype), _random(cols, 2, dtype)
    dy, dh = _random(h.shape, 3, dtype), _random(h.shape, 4, dtype)
    rstd = torch.empty(1100, device="cuda")
    F.flashopt_rms_norm(h, gain, rstd=rstd)
    want, want_gain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dh)
    for over in (0, 1):
        d = [dy.clone(), dh.clone()]
        dx, dgain = F.flashopt_rms_norm_backward(d[0], h, gain, rstd, d[1], dx=d[over])
        assert dx is d[over] and torch.equal(dx, want) and torch.equal(dgain, want_gain)
        assert torch.equal(d[1 - over], (dh, dy)[over])
    want, _ = F.flashopt_rms_norm_backward(dy, h, gain, rstd, dy.clone())
    both = dy.clone()
    F.flashopt_rms_norm_backward(both, h, gain, rstd, both, dx=both)
    assert torch.equal(both, want)


@pytest.mark.parametrize("shape", [(6, 300), (2, 3, 512)])
def test_broadcast_and_transposed_operands(shape):
    """Gradients of a plain sum (stride 0 throughout), rows and residuals that
    repeat one row, transposed inputs, and x as its own residual: as with copies
    in rows."""
    require_gpu()
    cols, w = shape[-1], _random((200, shape[-1]), 1, BF16)
    gain = _random(cols, 2, F32)

    def norm(x, residual, g, _):
        return F.rms_norm(x, g, residual)

    def linear(x, residual, g, weight):
        return F.fp8_norm_linear(x, g, weight, residual)

    def product(x, residual, g, weight):
        return (F.fp8_linear(x, weight),)
    x = _random(shape, 3, BF16)
    row = _random((cols,), 4, BF16).expand(shape)
    turned = _random((*shape[:-2], cols, shape[-2]), 5, BF16).transpose(-1, -2)
    for call in (norm, linear, product):
        for residual in (None, row, turned) if call is not product else (None,):
            got = call(x, residual, gain, w)
            want = call(x, None if residual is None else residual.contiguous(), gain, w)
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        for first in (row, turned):
            assert all(torch.equal(a, b) for a, b in zip(call(first, x if call is not product else None, gain, w),
                                                         call(first.contiguous(), x if call is not product else None,
                                                              gain, w)))
        # the gradient of a sum against that of the same ones in memory
        for residual in (None, turned) if call is not product else (None,):
            results = []
            for dense in (False, True):
                leaf = x.clone().requires_grad_()
                outs = [o for o in call(leaf, residual, gain.clone().requires_grad_(), w.clone().requires_grad_())]
                if dense:
                    torch.autograd.backward(outs, [torch.ones_like(o).contiguous() for o in outs])
                else:
                    sum(o.sum() for o in outs).backward()
                results.append(leaf.grad)
            assert torch.equal(*results)
    for call in (norm, linear):
        a, b = x.clone().requires_grad_(), x.clone().requires_grad_()
        other = x.clone().requires_grad_()
        one, two = call(a, a, gain, w), call(b, other, gain, w)
        assert all(torch.equal(p, q) for p, q in zip(one, two))
        one[0].sum().backward()
        two[0].sum().backward()
        assert torch.equal(b.grad, other.grad) and torch.equal(a.grad, b.grad + other.grad)


def test_two_captured_graphs_replayed_in_turn():
    """Graphs of forward and backward calls share no workspace: replayed in turn
    and on two streams at once, with eager work between, each gives what its
    eager call gave."""
    require_gpu()
    cases = []
    for i, (rows, cols, n) in enumerate([(300, 1001, 130), (40, 4096, 512), (1, 2048, 300)]):
        x, res = _random((rows, cols), 2 * i, BF16), _random((rows, cols), 2 * i + 1, BF16)
        gain, dy = _random(cols, 10 + i, F32), _random((rows, cols), 20 + i, BF16)
        w = F.flashopt_byte_quantize(_random((n, cols), 30 + i, BF16))
        rstd = torch.empty(rows, device="cuda")

        def run(x=x, res=res, gain=gain, dy=dy, w=w, rstd=rstd):
            (q, t), h = F.flashopt_rms_norm(x, gain, res, output="both", rstd=rstd)
            dx, dgain = F.flashopt_rms_norm_backward(dy, h, gain, rstd, res)
            return (h, q.codes.view(torch.uint8), t.codes.view(torch.uint8), t.scales, dx, dgain,
                    F.flashopt_byte_product(q, w), F.flashopt_byte_linear(x, w))
        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        cases.append((graph, got, want, run))        # run: keeps the inputs, which replays read
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(4):
        for _, got, _, _ in cases:
            for t in got:
                t.zero_()
        torch.cuda.synchronize()
        for (graph, *_), stream in zip(cases, streams):
            with torch.cuda.stream(stream if turn % 2 else torch.cuda.current_stream()):
                graph.replay()
        torch.cuda.synchronize()
        for _, got, want, _ in cases:
            assert all(torch.equal(a, b) for a, b in zip(got, want)), turn
        F.flashopt_rms_norm_backward(*[_random((50, 700), 1, BF16)] * 2, _random(700, 2, F32),
                                     torch.ones(50, device="cuda"))
