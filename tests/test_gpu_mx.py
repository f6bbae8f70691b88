"""The MXFP4 codec, product and linear layer on the GPU.

Codes and scales are compared byte for byte with a 64-bit reference: scaling
by a power of two is exact, so each code is one rounding of a known quotient.
Products are compared exactly where every partial sum is a small multiple of a
power of two, which fp32 holds in any order; elsewhere each of the K additions
is off by at most 2^-23 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


# ------------------------------------------------------------- references

def _ref_quantize(x):
    """(codes [R, Cp / 2], scales [R, Cp / 32]) of a host matrix."""
    x = x.to(F64).numpy()
    rows, cols = x.shape
    x = np.pad(x, ((0, 0), (0, -cols % 128))).reshape(rows, -1, 32)
    top = np.abs(x).max(axis=2)                          # NaN propagates
    bad = ~np.isfinite(top)
    _, e = np.frexp(np.where(bad, 0.0, top))             # top = f 2^e, f in [1/2, 1)
    e = np.where(top == 0, -127, np.maximum(e - 1 - 2, -127))
    y = np.ldexp(np.where(bad[..., None], 0.0, x), -e[..., None])
    a = np.minimum(np.abs(y), 6.0)
    step = np.where(a < 2, 0.5, np.where(a < 4, 1.0, 2.0))
    v = np.minimum(np.rint(a / step) * step, 6.0)        # rint: half to even
    code = np.searchsorted(GRID, v) | (np.signbit(y) << 3)
    code = np.where(bad[..., None], 0, code).reshape(rows, -1).astype(np.uint8)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    return code[:, 0::2] | (code[:, 1::2] << 4), byte


def _ref_values(codes, scales, cols):
    """fp64 values of codes and scales (device tensors in, device tensor out)."""
    table = torch.tensor(np.concatenate([GRID, -GRID]), device=codes.device)
    v = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], 2).view(codes.shape[0], codes.shape[1] // 16, 32)
    b = scales.to(torch.int64)
    unit = ((b - 127 + 1023) << 52).view(F64)
    unit = torch.where(b == 255, torch.full_like(unit, float("nan")), unit)
    return (v * unit[..., None]).view(codes.shape[0], 2 * codes.shape[1])[:, :cols]


def _values(q):
    return _ref_values(q.codes, q.scales, q.cols)


def _check_codes(q, x):
    codes, scales = _ref_quantize(x.detach().cpu())
    assert (q.rows, q.cols) == tuple(x.shape)
    assert (q.scales.cpu().numpy().reshape(scales.shape) == scales).all()
    assert (q.codes.cpu().numpy().reshape(codes.shape) == codes).all()


def _random(rows, cols, seed, dtype, spread=6):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * 2.0 ** torch.randint(-spread, spread + 1, (rows, cols), generator=g)
    return x.to(dtype).cuda()


# ------------------------------------------------------------------- codec

SHAPES = [(1, 1), (1, 33), (3, 128), (31, 32), (32, 256), (33, 257), (127, 129), (128, 128), (130, 1030),
          (333, 1001), (1, 4096), (2050, 1), (513, 64)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize(rows, cols, dtype):
    require_gpu()
    x = _random(rows, cols, rows + cols, dtype)
    q, t = F.flashopt_mx_quantize(x, "both")
    _check_codes(q, x)
    _check_codes(t, x.t())
    for one, layout, y in ((q, "rows", x), (t, "cols", x.t())):
        alone = F.flashopt_mx_quantize(x, layout)
        assert torch.equal(alone.codes, one.codes) and torch.equal(alone.scales, one.scales)
        want = _values(one)
        for out in (F32, BF16):
            v = F.flashopt_mx_dequantize(one, out)
            assert v.dtype == out and torch.equal(v.double(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_every_rounding(dtype):
    """Every quotient near a boundary between codes, at scales across the
    range, both signs; zeros of both signs; groups of the smallest values."""
    require_gpu()
    mids = np.array([0.0, 0.25, 0.5, 0.75, 1.0, 1.25, 1.5, 1.75, 2.0, 2.5, 3.0, 3.5, 4.0, 5.0, 6.0, 7.0])
    eps = 2.0 ** -6 if dtype == BF16 else 2.0 ** -20
    q = np.concatenate([mids, mids * (1 + eps), mids * (1 - eps)])
    q = np.concatenate([q, -q])                                # 96 quotients, below 8
    rows = []
    for e in range(-126, 125):
        groups = np.zeros((4, 32))
        groups[:, 0] = 4.0                                     # fixes the scale at 2^e
        groups[:, 1:25] = q.reshape(4, 24)
        rows.append(np.ldexp(groups.reshape(-1), e))
    x = torch.tensor(np.stack(rows)).to(dtype).cuda()
    _check_codes(F.flashopt_mx_quantize(x), x)
    tiny = torch.tensor([k * 2.0 ** (-133 if dtype == BF16 else -149) for k in range(-64, 64)], dtype=F64)
    edge = torch.stack([tiny, tiny * 2, torch.zeros(128, dtype=F64), -torch.zeros(128, dtype=F64)])
    edge = edge.to(dtype).cuda()
    big = torch.full((1, 128), torch.finfo(dtype).max, dtype=dtype, device="cuda")
    big[0, 1::2] *= -1
    for y in (edge, big):
        for layout, z in (("rows", y), ("cols", y.t())):
            _check_codes(F.flashopt_mx_quantize(y, layout), z)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_non_finite(dtype):
    """A group with an infinity or NaN stands for NaN; its neighbours do not."""
    require_gpu()
    x = _random(70, 300, 5, dtype)
    x[3, 40], x[3, 299], x[69, 0], x[10, 64] = float("inf"), float("nan"), -float("inf"), float("nan")
    q, t = F.flashopt_mx_quantize(x, "both")
    _check_codes(q, x)
    _check_codes(t, x.t())
    v = F.flashopt_mx_dequantize(q)
    assert torch.isnan(v[3, 32:64]).all() and torch.isnan(v[3, 288:]).all() and torch.isnan(v[69, :32]).all()
    assert int(torch.isnan(v).sum()) == 32 + 12 + 32 + 32


def test_quantize_views():
    """Row strides, odd offsets, a row repeated by expand, outputs into views;
    what lies around an output stays as it was."""
    require_gpu()
    for dtype in (BF16, F32):
        base = _random(90, 411, 9, dtype)
        for view in (base[:, 1:300], base[7:, :128], base[::3, 8:200], base[5:6].expand(40, 411),
                     base[1:2, 3:4]):
            q, t = F.flashopt_mx_quantize(view, "both")
            _check_codes(q, view)
            _check_codes(t, view.t())
        q = F.flashopt_mx_quantize(base[:, :301])
        for first, width in ((0, 301), (1, 301), (8, 301)):
            wide = torch.full((90, 320), 77.0, dtype=dtype, device="cuda")
            F.flashopt_mx_dequantize(q, out=wide[:, first:first + width])
            assert torch.equal(wide[:, first:first + width].double(), _values(q))
            assert (wide[:, :first] == 77).all() and (wide[:, first + width:] == 77).all()
    with pytest.raises(ValueError, match="contiguous"):
        F.flashopt_mx_quantize(base.t())
    with pytest.raises(ValueError, match="bf16 or fp32"):
        F.flashopt_mx_quantize(base.half())


def test_empty():
    require_gpu()
    x = torch.zeros(0, 40, device="cuda")
    q, t = F.flashopt_mx_quantize(x, "both")
    assert F.flashopt_mx_dequantize(q).shape == (0, 40) and F.flashopt_mx_dequantize(t).shape == (40, 0)
    w = F.flashopt_mx_quantize(torch.ones(5, 40, device="cuda"))
    assert F.flashopt_mx_product(q, w).shape == (0, 5)
    z = F.flashopt_mx_quantize(torch.zeros(3, 0, device="cuda"))
    for n in (3, 40, 700):
        u = F.flashopt_mx_quantize(torch.zeros(n, 0, device="cuda"))
        assert torch.equal(F.flashopt_mx_product(u, z, F32), torch.zeros(n, 3, device="cuda"))
    assert torch.equal(F.flashopt_mx_linear(torch.zeros(4, 0, device="cuda"), z), torch.zeros(4, 3, device="cuda"))


# ----------------------------------------------------------------- product

def _pair(m, n, k, seed, low=127, high=128):
    """MXTensors of random codes and scale bytes in [low, high]."""
    g = torch.Generator().manual_seed(seed)

    def one(rows):
        blocks = (k + 127) // 128
        codes = torch.randint(0, 256, (rows, 64 * blocks), generator=g, dtype=torch.uint8)
        scales = torch.randint(low, high + 1, (rows, 4 * blocks), generator=g, dtype=torch.uint8)
        pad = torch.arange(128 * blocks) >= k
        codes = torch.where(pad[0::2], 0, codes & 15) | torch.where(pad[1::2], 0, codes >> 4 << 4)
        scales = torch.where(torch.arange(4 * blocks) * 32 >= k, 0, scales)
        return F.MXTensor(codes.to(torch.uint8).cuda().contiguous(), scales.to(torch.uint8).cuda().contiguous(),
                          rows, k)
    return one(m), one(n)


# each tile shape and both ends of its range, ragged in all three directions
PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 17, 129), (3, 100, 1000), (15, 33, 255), (16, 64, 4096), (17, 65, 384),
            (31, 300, 640), (32, 32, 32), (33, 64, 128), (40, 1, 100), (64, 64, 256), (65, 129, 333),
            (100, 1, 4096), (128, 128, 128), (200, 300, 500), (257, 513, 640), (1, 4099, 4096),
            (2000, 1800, 200), (1793, 2049, 384), (3600, 3900, 130), (4097, 3500, 512),
            # small tiles, every kind of end along K; rows that share a workgroup's K, at the rule's border
            (300, 1100, 1), (300, 1100, 100), (301, 1101, 129), (300, 1100, 256), (299, 1100, 384), (300, 1100, 640),
            (300, 1100, 897), (300, 1100, 1000), (70, 5000, 333), (33, 9000, 300), (1000, 40, 4100), (64, 2048, 500),
            (64, 2049, 500), (128, 2048, 700), (129, 2048, 700), (8192, 16, 300), (8193, 16, 300),
            # K in four shares: every kind of end of the last one, and one that is left without
            (300, 1100, 6017), (300, 1100, 6144), (300, 1101, 6272), (299, 1100, 6400), (300, 1100, 6500),
            (300, 1100, 6700), (301, 1100, 6912), (300, 1100, 7000), (130, 5000, 12300), (1024, 1024, 6200)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product_exact(m, n, k):
    """Scales 1 and 2: every product is a multiple of 1/4 of at most 144, and
    4096 of them sum to less than 2^24 quarters."""
    require_gpu()
    a, b = _pair(m, n, k, m * 7 + n)
    want = _values(a) @ _values(b).t()
    print(f"product {m} x {n} x {k}", flush=True)
    assert torch.equal(F.flashopt_mx_product(a, b, F32).double(), want)
    assert torch.equal(F.flashopt_mx_product(a, b), want.to(F32).to(BF16))


@pytest.mark.parametrize("m,n,k", [(1, 500, 4096), (20, 100, 777), (60, 80, 2048), (700, 900, 1500),
                                   (1800, 2000, 300), (3600, 4000, 520)])
def test_product_wide_scales(m, n, k):
    require_gpu()
    a, b = _pair(m, n, k, 3, 107, 147)
    va, vb = _values(a), _values(b)
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    out = F.flashopt_mx_product(a, b, F32).double()
    assert ((out - want).abs() <= (k + 8) * 2.0 ** -23 * size).all()


def test_product_far_scales():
    """Single groups at the ends of the range, and 2^-56 2^-56 and 2^56 2^56."""
    require_gpu()
    for low, high in ((71, 71), (183, 183), (1, 1), (0, 0), (250, 250)):
        a, b = _pair(5, 40, 32, 4, low, low)
        c, _ = _pair(5, 40, 32, 5, 254 - high, 254 - high)
        want = _values(c) @ _values(b).t()               # 2^e 2^-e: exact
        assert torch.equal(F.flashopt_mx_product(c, b, F32).double(), want), low
        if low in (71, 183):
            want = _values(a) @ _values(b).t()
            assert torch.equal(F.flashopt_mx_product(a, b, F32).double(), want), low


@pytest.mark.parametrize("m,n,k", [(4, 50, 300), (50, 70, 300), (2000, 1800, 200), (3600, 3900, 130), (300, 1100, 300),
                                   (300, 1100, 6200)])
def test_product_nan_scale(m, n, k):
    """A NaN scale reaches its row or column of the product and no other."""
    require_gpu()
    a, b = _pair(m, n, k, 6)
    a.scales[m // 2, 1] = 255
    b.scales[n - 1, 0] = 255
    b.codes[n - 1, :16] = 0
    for dtype in (F32, BF16):
        nan = torch.isnan(F.flashopt_mx_product(a, b, dtype))
        want = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        want[m // 2], want[:, n - 1] = True, True
        assert torch.equal(nan, want)


def test_product_into_views():
    """Rows of a wider output, aligned and not; what lies around stays."""
    require_gpu()
    for m, n, k in ((5, 45, 200), (70, 90, 200), (2000, 1801, 128), (3600, 3901, 128)):
        a, b = _pair(m, n, k, 8)
        want = _values(a) @ _values(b).t()
        for dtype in (F32, BF16):
            for first in (0, 1, 4):
                wide = torch.full((m, n + 11), 3.0, dtype=dtype, device="cuda")
                F.flashopt_mx_product(a, b, out=wide[:, first:first + n])
                assert torch.equal(wide[:, first:first + n], want.to(F32).to(dtype))
                assert (wide[:, :first] == 3).all() and (wide[:, first + n:] == 3).all()


def test_offsets_past_32_bits():
    """Matrices, codes and outputs of more than 2^32 bytes and elements: the
    far end equals the same rows on their own, and a product there is exact
    (small integers: every sum is)."""
    require_gpu()
    rows, cols, tail = 70_000, 131_072, 300
    x = torch.zeros(rows, cols, dtype=BF16, device="cuda")           # 18 GB, codes of 4.6 GB
    g = torch.Generator(device="cuda").manual_seed(3)
    x[-tail:] = torch.randint(-3, 4, (tail, cols), generator=g, device="cuda", dtype=torch.int32).to(BF16)
    q, t = F.flashopt_mx_quantize(x, "both")
    end = F.flashopt_mx_quantize(x[-tail:])
    assert torch.equal(q.codes[-tail:], end.codes) and torch.equal(q.scales[-tail:], end.scales)
    right = F.flashopt_mx_quantize(x[:, -256:], "cols")
    assert torch.equal(t.codes[-256:], right.codes) and torch.equal(t.scales[-256:], right.scales)
    wide = F.flashopt_mx_dequantize(q, BF16)
    assert torch.equal(wide[-tail:], F.flashopt_mx_dequantize(end, BF16))
    assert not wide[:4].any() and not wide[-tail - 4:-tail].any()
    del wide, t, right, x
    for m in (3, 40):                                                # few rows, tiles
        a = F.flashopt_mx_quantize(_random(m, cols, 4, BF16, 0).round().clamp(-2, 2))
        out = F.flashopt_mx_product(a, q, F32)
        want = _values(a) @ _values(end).t()
        assert torch.equal(out[:, -tail:], want.to(F32)), m
        assert not out[:, :rows - tail].any()
    del q, end, out, want
    # an output of 4.6 G elements
    n = 68_000
    x = torch.randint(-3, 4, (n, 128), generator=g, device="cuda", dtype=torch.int32).to(BF16)
    q = F.flashopt_mx_quantize(x)
    out = F.flashopt_mx_product(q, q)
    v = _values(q)
    for at in (0, 31_000, n - 500):
        want = v[at:at + 500] @ v.t()
        assert torch.equal(out[at:at + 500], want.to(BF16)), at


# ------------------------------------------------------------------ linear

def test_linear_equals_quantize_and_product():
    require_gpu()
    # up to four aligned rows of bf16 are quantized inside the product
    for m, n, k in ((1, 300, 500), (1, 300, 504), (3, 9000, 4096), (4, 8200, 24), (4, 17, 264), (1, 5, 8),
                    (16, 64, 4096), (17, 40, 130), (200, 100, 64), (2100, 2048, 256)):
        for dtype in (BF16, F32):
            x, w = _random(m, k, 1, dtype, 2), F.flashopt_mx_quantize(_random(n, k, 2, BF16, 2))
            for out in (BF16, F32):
                y = F.flashopt_mx_linear(x, w, out)
                assert torch.equal(y, F.flashopt_mx_product(F.flashopt_mx_quantize(x), w, out))
    x, w = _random(2, 4096, 5, BF16), F.flashopt_mx_quantize(_random(50, 4096, 6, BF16, 2))
    x[1, 70], x[1, 4000] = float("nan"), float("inf")
    y = F.flashopt_mx_linear(x, w, F32)
    assert torch.equal(y[0], F.flashopt_mx_linear(x[:1], w, F32)[0]) and torch.isnan(y[1]).all()
    assert torch.isfinite(y[0]).all()
    wide = _random(40, 300, 3, BF16)
    w = F.flashopt_mx_quantize(_random(33, 200, 4, BF16))
    for view in (wide[:3, 8:208], wide[:3, 7:207], wide[4:5, 96:296], wide[2:3, :200].expand(4, 200)):
        assert torch.equal(F.flashopt_mx_linear(view, w), F.flashopt_mx_linear(view.contiguous(), w))
    view = wide[:, 7:207]
    assert torch.equal(F.flashopt_mx_linear(view, w), F.flashopt_mx_linear(view.contiguous(), w))
    with pytest.raises(ValueError, match="columns"):
        F.flashopt_mx_linear(wide, w)
    with pytest.raises(F.FlashoptError, match="EWORKSPACE"):
        F.flashopt_mx_linear(view, w, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


def test_linear_on_both_sides_of_its_rule():
    """Few rows and a weight of 2^26 elements, and more: in one launch and in
    two, the same values."""
    require_gpu()
    g = torch.Generator(device="cuda").manual_seed(9)
    for n in ((1 << 26) // 4096, (1 << 26) // 4096 + 1):
        w = F.flashopt_mx_quantize(torch.randn(n, 4096, generator=g, device="cuda"))
        for m in (1, 4, 5):
            x = _random(m, 4096, m, BF16, 2)
            assert torch.equal(F.flashopt_mx_linear(x, w), F.flashopt_mx_product(F.flashopt_mx_quantize(x), w))


@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape,n", [((5,), 40), ((1, 64), 33), ((3, 17, 100), 64), ((300, 257), 129), ((0, 8), 4)])
def test_mx_linear_gradients(shape, n, dtype, held):
    """Forward and gradients are the products of the quantized operands,
    each grouped along the axis it is summed over."""
    require_gpu()
    k = shape[-1]
    x = _random(int(np.prod(shape[:-1])), k, 1, dtype, 2).view(shape).requires_grad_()
    w = _random(n, k, 2, dtype, 2).requires_grad_()
    weight = F.MXWeight(w) if held else w
    y = F.mx_linear(x, weight)
    dy = _random(int(np.prod(shape[:-1])), n, 3, dtype, 2).view(*shape[:-1], n)
    dx, dw = torch.autograd.grad(y, (x, w), dy)
    assert y.shape == dy.shape and dx.shape == x.shape and dw.shape == w.shape
    flat, dflat = x.detach().reshape(-1, k) if x.numel() else x.detach(), dy.reshape(-1, n) if dy.numel() else dy
    q = lambda t, layout="rows": _values(F.flashopt_mx_quantize(t.detach(), layout))
    for got, left, right in ((y, q(flat), q(w)), (dx, q(dflat), q(w, "cols")),
                             (dw, q(dflat, "cols"), q(flat, "cols"))):
        want, size = left @ right.t(), left.abs() @ right.abs().t()
        # K additions in fp32, and one rounding to the type
        bound = (left.shape[1] + 8) * 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * want.abs() * (1 + 2 ** -8)
        assert got.dtype == dtype
        assert ((got.detach().reshape(want.shape).double() - want).abs() <= bound).all()


def test_mx_linear_differences():
    """On matrices that quantize to themselves the layer is bilinear, and its
    gradients are its differences, exactly: small integers throughout."""
    require_gpu()
    g = torch.Generator().manual_seed(0)

    def grid(rows, cols):      # values of the grid; a 6 in each group of either direction
        v = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0])[torch.randint(0, 6, (rows, cols), generator=g)]
        v *= torch.randint(0, 2, (rows, cols), generator=g) * 2 - 1
        i, j = torch.arange(rows)[:, None], torch.arange(cols)
        return torch.where((i + j) % 32 == 0, 6.0, v).cuda()
    x, w, dy = grid(64, 96), grid(128, 96), grid(64, 128)
    x.requires_grad_()
    w.requires_grad_()
    dx, dw = torch.autograd.grad(F.mx_linear(x, w), (x, w), dy)
    with torch.no_grad():
        base = (F.mx_linear(x, w) * dy).sum(dtype=F64)
        for t, grad, at in ((x, dx, [(0, 1), (5, 40), (63, 95)]), (w, dw, [(0, 1), (77, 3), (127, 95)])):
            for i, j in at:
                old = float(t[i, j])
                new = 1.0 if old != 1.0 else -2.0
                t[i, j] = new
                diff = (F.mx_linear(x, w) * dy).sum(dtype=F64) - base
                t[i, j] = old
                assert float(diff) == float(grad[i, j]) * (new - old)


def test_mx_linear_partial_gradients_and_versions():
    require_gpu()
    x, w = _random(40, 100, 1, BF16), _random(50, 100, 2, BF16)
    dy = _random(40, 50, 3, BF16)
    xr, wr = x.clone().requires_grad_(), w.clone().requires_grad_()
    both = torch.autograd.grad(F.mx_linear(xr, wr), (xr, wr), dy)
    assert torch.equal(torch.autograd.grad(F.mx_linear(xr, w), xr, dy)[0], both[0])
    assert torch.equal(torch.autograd.grad(F.mx_linear(x, wr), wr, dy)[0], both[1])
    xr.grad = None
    F.mx_linear(xr, wr).float().sum().backward()           # an expanded output gradient
    ones = torch.autograd.grad(F.mx_linear(xr, wr), xr, torch.ones_like(dy))[0]
    assert torch.equal(xr.grad, ones)
    weight = F.MXWeight(wr)
    y = F.mx_linear(xr, weight)
    with torch.no_grad():
        wr.mul_(2)
    assert torch.equal(F.mx_linear(x, weight), y)          # the copies follow refresh()
    weight.refresh()
    assert torch.equal(F.mx_linear(x, weight), F.mx_linear(x, wr))
    with pytest.raises(RuntimeError, match="refreshed"):
        y.backward(dy)


def test_other_stream_and_graph():
    """On a side stream, and captured: replays with new inputs, eager work
    between them."""
    require_gpu()
    side = torch.cuda.Stream()
    w = F.MXWeight(_random(300, 200, 1, BF16, 2))
    x = _random(60, 200, 2, BF16, 2)
    want = F.flashopt_mx_linear(x, w.rows)
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        q = F.flashopt_mx_quantize(x, stream=stream)
        outs = [F.flashopt_mx_product(q, w.rows, stream=stream), F.flashopt_mx_linear(x, w.rows, stream=stream)]
        side.synchronize()
        assert all(torch.equal(o, want) for o in outs)
    buf, p = torch.zeros_like(x), w.param.clone()
    held = F.MXWeight(p)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.refresh()
        q, t = F.flashopt_mx_quantize(buf, "both")
        outs = [F.flashopt_mx_linear(buf, held.rows), F.flashopt_mx_product(t, t, F32),
                F.flashopt_mx_dequantize(q)]
    for i in range(4):
        buf.copy_(_random(60, 200, 10 + i, BF16, 2))
        p.copy_(_random(300, 200, 20 + i, BF16, 2))
        graph.replay()
        q, t = F.flashopt_mx_quantize(buf, "both")
        eager = [F.flashopt_mx_linear(buf, F.flashopt_mx_quantize(p)), F.flashopt_mx_product(t, t, F32),
                 F.flashopt_mx_dequantize(q)]
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            assert torch.equal(o, e), i


# ---------------------------------------------------- the operators together

def test_captured_training_step():
    """Forward, backward, norm, clipped step and requantization in one graph;
    replays with new inputs, eager steps of a second copy between them, equal
    bits.  The captured parameter is in no eager graph."""
    require_gpu()
    rows, cols = 130, 200
    pa, pb = [W.init_param(rows * cols, device="cuda", seed=3).view(rows, cols).requires_grad_() for _ in range(2)]
    a, b = [F.FlashAdamW([p.detach()], **W.HP_DEFAULT) for p in (pa, pb)]
    wa, wb = F.MXWeight(pa), F.MXWeight(pb)
    x, dy = torch.zeros(70, cols, dtype=BF16, device="cuda"), torch.zeros(70, rows, dtype=BF16, device="cuda")
    grad, out = torch.zeros(rows, cols, dtype=BF16, device="cuda"), torch.zeros(2, device="cuda")
    norm, plan = F.GradPlan([grad]), a.plan([grad], step=1, grad_scale=out[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = F.mx_linear(x, wa)
        grad.copy_(torch.autograd.grad(y, [pa], dy)[0])
        y = y.detach()
        norm.norm(0.01, out=out)
        plan.launch()
        wa.refresh()
    for t in (1, 2, 3, 4):
        x.copy_(_random(70, cols, t, BF16, 1))
        dy.copy_(_random(70, rows, 40 + t, BF16, 1) * 1e-2)
        plan.set_step(t)
        graph.replay()
        z = F.mx_linear(x, wb)
        z.backward(dy)
        eager = b.step([pb.grad], max_norm=0.01)
        pb.grad = None
        wb.refresh()
        torch.cuda.synchronize()
        assert torch.equal(y, z) and torch.equal(out, eager) and float(out[1]) < 1.0, t
        assert torch.equal(pa, pb) and torch.equal(a.states[0].block, b.states[0].block), t
        for q, r in ((wa.rows, wb.rows), (wa.cols, wb.cols)):
            assert torch.equal(q.codes, r.codes) and torch.equal(q.scales, r.scales), t


@pytest.mark.parametrize("release", [False, True])
def test_training_steps(release):
    """MXFP4 layers, the clipped step on compressed states and new copies of
    the weights, for three steps; a second run from the same parts agrees bit
    for bit.  With gradient release, the hooks step each weight."""
    require_gpu()
    shapes = [(160, 96), (64, 160)]

    def run():
        params = [W.init_param(a * b, device="cuda", seed=i).view(a, b).requires_grad_()
                  for i, (a, b) in enumerate(shapes)]
        opt = F.FlashAdamW([p.detach() for p in params], **W.HP_DEFAULT)
        weights = [F.MXWeight(p) for p in params]
        handles = F.attach_grad_release(opt, params, batch_below=0) if release else []
        seen = []
        for t in (1, 2, 3):
            x = _random(48, 96, t, BF16, 1)
            h = torch.relu(F.mx_linear(x, weights[0]))
            y = F.mx_linear(h, weights[1])
            y.backward(_random(48, 64, 50 + t, BF16, 1) * 1e-2)
            if not release:
                grads = [p.grad for p in params]
                out = opt.step([g for g in grads], max_norm=0.01)
                assert float(out[1]) < 1.0
                assert torch.equal(out, F.flashopt_grad_norm(grads, 0.01))
                seen.append(out.clone())
            for p, w in zip(params, weights):
                assert not release or p.grad is None
                p.grad = None
                w.refresh()
                _check_codes(w.rows, p)
                _check_codes(w.cols, p.t())
            seen += [y.detach().clone()] + [p.detach().clone() for p in params]
        for h in handles:
            h.remove()
        assert not torch.equal(seen[-1], W.init_param(64 * 160, device="cuda", seed=1).view(64, 160))
        return seen
    for a, b in zip(run(), run()):
        assert torch.equal(a, b)
