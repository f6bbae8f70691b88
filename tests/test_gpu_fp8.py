"""The 8-bit codec, product and linear layer on the GPU.

Codes and scales are compared byte for byte with a 64-bit reference: scaling
by a power of two is exact, so each code is one rounding of a known quotient.
Products are compared exactly where every partial sum is a small multiple of a
power of two, which fp32 holds in any order.  Elsewhere two errors count.  The
matrix instructions align the products of eight consecutive k to the largest
one and drop what lies 2^-13 below its binade (the product of the two values'
powers of two; test_octets holds that bit for bit), so an octet is off by less
than 7 x 2^-13 of that power.  And each of the K additions in fp32 is off by at
most 2^-24 of the sum of magnitudes, or 2^-23 if it truncates."""
import numpy as np
import pytest
import torch

from bit_companded_adam_amd import flashopt as F
from bit_companded_adam_amd import workloads as W
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
# mantissa bits, exponent of the smallest normal value, exponent of the top binade
KIND = {E4M3: (3, -6, 8), E5M2: (2, -14, 15)}


# ------------------------------------------------------------- references

def _ref_quantize(x, dtype, block=False):
    """(codes [R, Cp] uint8, scales [R, groups padded to 16]) of a host matrix."""
    bits, low, top_exp = KIND[dtype]
    x = x.to(F64).numpy()
    rows, cols = x.shape
    x = np.pad(x, ((0, -rows % 128), (0, -cols % 128)))
    g = x.reshape(x.shape[0] // 128, 128, x.shape[1] // 128, 128)
    top = np.abs(g).max(axis=(1, 3) if block else 3, keepdims=True)     # NaN propagates
    bad = ~np.isfinite(top)
    f, e = np.frexp(np.where(bad, 0.0, top))             # top = f 2^e, f in [1/2, 1)
    e = np.where(top == 0, -127, np.maximum(e - 1 - top_exp + (f > 0.875), -127))
    y = np.ldexp(np.where(bad, 0.0, g), -e)
    _, b = np.frexp(np.abs(y))
    step = np.ldexp(1.0, np.maximum(b - 1, low) - bits)
    v = np.rint(y / step) * step                         # rint: half to even
    assert np.abs(v).max(initial=0) <= 1.75 * 2.0 ** top_exp
    codes = torch.from_numpy(np.where(bad, 0.0, v)).float().to(dtype)   # exact: these are the format's values
    assert (codes.to(F64).numpy() == np.where(bad, 0.0, v)).all()
    byte = np.broadcast_to(np.where(bad, 255, e + 127), (g.shape[0], 128, g.shape[2], 1)).astype(np.uint8)
    byte = byte.reshape(x.shape[0], -1)[:rows]
    return (codes.view(torch.uint8).numpy().reshape(x.shape)[:rows],
            np.pad(byte, ((0, 0), (0, -byte.shape[1] % 16))))


def _values(q):
    """fp64 values of an FP8Tensor's codes and scales."""
    b = q.scales[:, :q.codes.shape[1] // 128].to(torch.int64)
    unit = ((b - 127 + 1023) << 52).view(F64)
    unit = torch.where(b == 255, torch.full_like(unit, float("nan")), unit)
    return (q.codes.to(F64).view(q.rows, -1, 128) * unit[..., None]).view(q.rows, -1)[:, :q.cols]


def _check_codes(q, x, dtype=E4M3, block=False):
    codes, scales = _ref_quantize(x.detach().cpu(), dtype, block)
    assert (q.rows, q.cols, q.dtype) == (*x.shape, dtype)
    assert (q.scales.cpu().numpy() == scales).all()
    assert (q.codes.view(torch.uint8).cpu().numpy() == codes).all()


def _random(rows, cols, seed, dtype, spread=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * 2.0 ** torch.randint(-spread, spread + 1, (rows, cols), generator=g)
    return x.to(dtype).cuda()


# ------------------------------------------------------------------- codec

SHAPES = [(1, 1), (1, 33), (3, 128), (31, 32), (32, 256), (33, 257), (127, 129), (128, 128), (129, 127), (130, 1030),
          (333, 1001), (1, 4096), (2050, 1), (513, 64), (300, 2049), (4097, 130)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
@pytest.mark.parametrize("block", [False, True])
def test_quantize(rows, cols, dtype, kind, block):
    require_gpu()
    x = _random(rows, cols, rows + cols, dtype, 8 if kind == E4M3 else 16)
    q, t = F.flashopt_byte_quantize(x, "both", block, kind)
    _check_codes(q, x, kind, block)
    _check_codes(t, x.t(), kind, block)
    if block:
        assert torch.equal(_values(q), _values(t).t())
    for one, layout in ((q, "rows"), (t, "cols")):
        alone = F.flashopt_byte_quantize(x, layout, block, kind)
        assert torch.equal(alone.codes.view(torch.uint8), one.codes.view(torch.uint8))
        assert torch.equal(alone.scales, one.scales)
        want = _values(one)
        for out in (F32, BF16):
            v = F.flashopt_byte_dequantize(one, out)
            assert v.dtype == out and torch.equal(v.double(), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_quantize_every_rounding(dtype, kind):
    """Every quotient near a boundary between codes, at scales across the
    range, both signs; the largest values that one scale takes and the next
    ones up; groups of the smallest values and of zeros of both signs."""
    require_gpu()
    top_exp = KIND[kind][2]
    top = 1.75 * 2.0 ** top_exp
    codes = torch.arange(0, 256, dtype=torch.uint8).view(kind).double()
    codes = np.unique(codes[torch.isfinite(codes) & (codes >= 0)].numpy())
    assert codes[-1] == top
    mids = np.concatenate([codes, (codes[1:] + codes[:-1]) / 2])
    eps = 2.0 ** -7 if dtype == BF16 else 2.0 ** -20
    q = np.concatenate([mids, mids * (1 + eps), mids * (1 - eps)])
    q = np.concatenate([q[q <= top], -q[q <= top]])
    q = np.pad(q, (0, -len(q) % 127)).reshape(-1, 127)
    q = np.concatenate([np.full((len(q), 1), top), q], axis=1).reshape(-1)     # the first fixes the scale
    lowest = -126 + KIND[kind][0] - KIND[kind][1]          # every quotient is a normal fp32
    rows = [np.ldexp(q, e) for e in [*range(lowest, 126 - top_exp, 7), 126 - top_exp]]
    x = torch.tensor(np.stack(rows)).to(dtype).cuda()
    for layout, y in (("rows", x), ("cols", x.t())):
        _check_codes(F.flashopt_byte_quantize(x, layout, dtype=kind), y, kind)
    # the border between scales: 1.75 2^e and its neighbours, and the last few
    # scales at both ends
    border = []
    for e in [*range(-133, -100), *range(-3, 4), *range(100, 128)]:
        one = torch.tensor([1.75 * 2.0 ** e]).to(dtype)
        bits = one.view(torch.int16 if dtype == BF16 else torch.int32)
        near = torch.cat([bits - 1, bits, bits + 1]).view(dtype)
        border.append(torch.cat([near[:, None], near[:, None] * -0.3, near[:, None] * 0.001, torch.zeros(3, 125)], 1))
    border = torch.cat([b.to(dtype) for b in border])
    tiny = torch.tensor([k * 2.0 ** (-133 if dtype == BF16 else -149) for k in range(-64, 64)], dtype=F64)
    edge = torch.stack([tiny, tiny * 2, tiny * 2.0 ** 9, torch.zeros(128, dtype=F64), -torch.zeros(128, dtype=F64)])
    big = torch.full((1, 128), torch.finfo(dtype).max, dtype=dtype)
    big[0, 1::2] *= -1
    for y in (border.cuda(), edge.to(dtype).cuda(), big.cuda()):
        for layout, z in (("rows", y), ("cols", y.t())):
            for block in (False, True):
                _check_codes(F.flashopt_byte_quantize(y, layout, block, kind), z, kind, block)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_quantize_non_finite(dtype, kind):
    """A group with an infinity or NaN stands for NaN; its neighbours do not."""
    require_gpu()
    x = _random(150, 300, 5, dtype)
    x[3, 40], x[3, 299], x[149, 0], x[10, 140] = float("inf"), float("nan"), -float("inf"), float("nan")
    q, t = F.flashopt_byte_quantize(x, "both", dtype=kind)
    _check_codes(q, x, kind)
    _check_codes(t, x.t(), kind)
    alone = F.flashopt_byte_quantize(x, dtype=kind)
    assert torch.equal(alone.codes.view(torch.uint8), q.codes.view(torch.uint8)) and torch.equal(alone.scales, q.scales)
    v = F.flashopt_byte_dequantize(q)
    assert int(torch.isnan(v).sum()) == 128 + 44 + 128 + 128
    q, t = F.flashopt_byte_quantize(x, "both", True, kind)
    _check_codes(q, x, kind, True)
    _check_codes(t, x.t(), kind, True)


def test_quantize_views():
    """Row strides, odd offsets, a row repeated by expand, outputs into views;
    what lies around an output stays as it was."""
    require_gpu()
    for dtype in (BF16, F32):
        base = _random(190, 411, 9, dtype)
        for view in (base[:, 1:300], base[7:, :128], base[::3, 8:200], base[5:6].expand(40, 411),
                     base[1:2, 3:4], base[2:150, 3:300]):
            q, t = F.flashopt_byte_quantize(view, "both")
            _check_codes(q, view)
            _check_codes(t, view.t())
            _check_codes(F.flashopt_byte_quantize(view), view)
            _check_codes(F.flashopt_byte_quantize(view, block=True), view, block=True)
        q = F.flashopt_byte_quantize(base[:, :301])
        for first, width in ((0, 301), (1, 301), (8, 301)):
            wide = torch.full((190, 320), 77.0, dtype=dtype, device="cuda")
            F.flashopt_byte_dequantize(q, out=wide[:, first:first + width])
            assert torch.equal(wide[:, first:first + width].double(), _values(q))
            assert (wide[:, :first] == 77).all() and (wide[:, first + width:] == 77).all()
    with pytest.raises(ValueError, match="contiguous"):
        F.flashopt_byte_quantize(base.t())
    with pytest.raises(ValueError, match="bf16 or fp32"):
        F.flashopt_byte_quantize(base.half())


@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_dequantize_every_code(kind):
    """Every code under every scale, NaN codes (and E5M2's infinities) too: fp32
    holds each product up to its largest value; bf16 is its rounding."""
    require_gpu()
    codes = torch.arange(256, dtype=torch.uint8).view(1, 256).repeat(256, 1)
    scales = torch.zeros(256, 16, dtype=torch.uint8)
    scales[:, 0] = scales[:, 1] = torch.arange(256)
    q = F.FP8Tensor(codes.cuda().view(kind), scales.cuda(), 256, 256)
    want = _values(q)
    for out in (F32, BF16):
        got = F.flashopt_byte_dequantize(q, out)
        torch.testing.assert_close(got, want.to(F32).to(out), rtol=0, atol=0, equal_nan=True)


def test_empty():
    require_gpu()
    x = torch.zeros(0, 40, device="cuda")
    q, t = F.flashopt_byte_quantize(x, "both")
    assert F.flashopt_byte_dequantize(q).shape == (0, 40) and F.flashopt_byte_dequantize(t).shape == (40, 0)
    w = F.flashopt_byte_quantize(torch.ones(5, 40, device="cuda"))
    assert F.flashopt_byte_product(q, w).shape == (0, 5)
    z = F.flashopt_byte_quantize(torch.zeros(3, 0, device="cuda"))
    for n in (3, 40, 700):
        u = F.flashopt_byte_quantize(torch.zeros(n, 0, device="cuda"))
        assert torch.equal(F.flashopt_byte_product(u, z, F32), torch.zeros(n, 3, device="cuda"))
    assert torch.equal(F.flashopt_byte_linear(torch.zeros(4, 0, device="cuda"), z), torch.zeros(4, 3, device="cuda"))


# ----------------------------------------------------------------- product

def _pair(m, n, k, seed, kind=E4M3, low=127, high=128, small=True):
    """FP8Tensors of random codes (small: integers of at most 8) and scale bytes
    in [low, high]."""
    g = torch.Generator().manual_seed(seed)

    def one(rows, dtype):
        blocks = (k + 127) // 128
        if small:
            codes = torch.randint(-8, 9, (rows, 128 * blocks), generator=g).float()
            codes = codes.to(dtype)          # three bits hold them
        else:
            codes = torch.randint(0, 256, (rows, 128 * blocks), generator=g, dtype=torch.uint8).view(dtype)
            codes = torch.where(torch.isfinite(codes.float()), codes.float(), torch.zeros(())).to(dtype)
        codes = torch.where(torch.arange(128 * blocks) >= k, torch.zeros(()), codes.float()).to(dtype)
        scales = torch.zeros(rows, (blocks + 15) // 16 * 16, dtype=torch.uint8)
        scales[:, :blocks] = torch.randint(low, high + 1, (rows, blocks), generator=g, dtype=torch.uint8)
        return F.FP8Tensor(codes.cuda().contiguous(), scales.cuda(), rows, k)
    return one(m, kind), one(n, E4M3)


# each tile shape and both ends of its range, ragged in all three directions
PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 17, 129), (3, 100, 1000), (15, 33, 255), (16, 64, 4096), (17, 65, 384),
            (31, 300, 640), (32, 32, 32), (33, 64, 128), (40, 1, 100), (64, 64, 256), (65, 129, 333),
            (100, 1, 4096), (128, 128, 128), (200, 300, 500), (257, 513, 640), (1, 4099, 4096),
            (2000, 1800, 200), (1793, 2049, 384), (3600, 3900, 130), (4097, 3500, 512),
            (300, 1100, 1), (300, 1100, 100), (301, 1101, 129), (300, 1100, 256), (299, 1100, 384), (300, 1100, 640),
            (300, 1100, 897), (300, 1100, 1000), (70, 5000, 333), (33, 9000, 300), (1000, 40, 4100), (64, 2048, 500),
            (64, 2049, 500), (128, 2048, 700), (129, 2048, 700), (8192, 16, 300), (8193, 16, 300),
            # scales past the first sixteen of a row, every kind of end
            (300, 1100, 1920), (300, 1100, 2048), (300, 1101, 2176), (299, 1100, 2200), (300, 1100, 4096),
            (300, 1100, 4224), (130, 5000, 12300), (1024, 1024, 6200), (2100, 2100, 2300), (4000, 3800, 4200),
            # one row: pieces of 1024, shares of a few steps, more rows of B than one grid takes
            (1, 300, 1), (1, 301, 1023), (1, 1, 1024), (1, 33, 1025), (1, 100, 4096), (1, 50, 5000), (1, 2200001, 128),
            # few rows or tiles, each shape: ends of the fours of steps that a wavefront takes, of the 128 whose
            # scales are held, and shares that are left without any
            (2, 40, 128), (2, 40, 256), (3, 40, 384), (5, 40, 512), (16, 40, 640), (9, 700, 2048), (2, 30, 2176),
            (7, 30, 16384), (7, 33, 16385), (16, 17, 16512), (11, 40, 33000), (20, 4096, 300), (33, 4096, 1000),
            (33, 4097, 900), (16, 6000, 500), (15, 14336, 400), (2, 20000, 200), (40, 5000, 700), (48, 9000, 260),
            (64, 9000, 260), (30, 9000, 260), (128, 4096, 520), (129, 4096, 520), (250, 4000, 2048), (250, 4000, 2047),
            (64, 20000, 130), (33, 17000, 130)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_product_exact(m, n, k, kind):
    """Integers of at most 64 x 4 in each term: every partial sum up to K = 65536
    is an integer below 2^24, which fp32 holds."""
    require_gpu()
    a, b = _pair(m, n, k, m + n + k, kind)
    want = _values(a) @ _values(b).t()
    got = F.flashopt_byte_product(a, b, F32)
    assert torch.equal(got.double(), want)
    got = F.flashopt_byte_product(a, b)
    assert got.dtype == BF16 and torch.equal(got, want.float().to(BF16))


def _binade(v):
    """The power of two at or below a magnitude (0 for 0)."""
    _, e = torch.frexp(v.abs())
    return torch.where(v == 0, torch.zeros_like(v), torch.ldexp(torch.ones_like(v), e - 1))


def _off(va, vb):
    """The most that each output of a product may be off by, in fp32."""
    k = va.shape[1]
    pad = torch.nn.functional.pad
    pa, pb = [pad(_binade(v), (0, -k % 8)).view(v.shape[0], -1, 8) for v in (va, vb)]
    octets = torch.zeros(va.shape[0], vb.shape[0], dtype=F64, device=va.device)
    for i in range(pa.shape[1]):
        octets += (pa[:, None, i] * pb[None, :, i]).amax(2)
    return octets * 7 * 2.0 ** -13 + va.abs() @ vb.abs().t() * k * 2.0 ** -23


def _check_product(got, va, vb):
    """A product against 64 bits: a sample of its rows and columns, the corners
    among them, to the octets' bound; all of it to the sum of magnitudes times
    2^-10, which that is below."""
    half = torch.finfo(got.dtype).eps / 2
    want, size = va @ vb.t(), va.abs() @ vb.abs().t()
    bound = size * (2.0 ** -10 + va.shape[1] * 2.0 ** -23)
    assert ((got.double() - want).abs() <= bound + (want.abs() + bound) * half).all()
    i, j = [torch.linspace(0, n - 1, min(n, most), device=va.device).round().long()
            for n, most in ((va.shape[0], 24), (vb.shape[0], 128))]
    want, bound = want[i][:, j], _off(va[i], vb[j])
    assert ((got.double()[i][:, j] - want).abs() <= bound + (want.abs() + bound) * half).all()


@pytest.mark.parametrize("m,n,k", [(5500, 2001, 300), (3201, 3329, 136), (2700, 4100, 2100), (3840, 2560, 128),
                                   (4033, 4600, 1)])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_product_exact_in_lower_tiles(m, n, k, kind):
    """Sizes whose 256 x 256 tiles would leave CUs idle: tiles of 192 rows of a."""
    test_product_exact(m, n, k, kind)


def test_octets():
    """What the instructions keep of eight products: those above 2^-13 of the
    largest one's binade, each cut there toward zero; across octets it is 2^-24
    of it, fp32's own."""
    require_gpu()
    for m, n in ((16, 16), (300, 1100)):
        va, vb = torch.zeros(m, 128), torch.zeros(n, 128)
        va[0, 0], va[0, 1], vb[0, 0], vb[0, 1] = 256, 256, 256, -256       # cancel
        want = []
        for i in range(1, 16):
            va[i], vb[i] = va[0], vb[0]
            vb[i, 2 + (i & 4)], va[i, 2 + (i & 4)] = 1.0, i
            va[i, 8 + (i & 4)], vb[i, 8 + (i & 4)] = 2.0 ** -4, 2.0 ** -4  # the next octet
            want.append((i // 8 * 8) + 2.0 ** -8)
        a, b = [F.flashopt_byte_quantize(torch.cat([v, torch.full((v.shape[0], 128), 448.0)], 1).cuda()) for v in (va, vb)]
        a.scales[:, :2], b.scales[:, :2] = 127, 127
        a.codes.view(torch.uint8)[:, :128] = va.to(E4M3).view(torch.uint8).cuda()
        b.codes.view(torch.uint8)[:, :128] = vb.to(E4M3).view(torch.uint8).cuda()
        a.codes.view(torch.uint8)[:, 128:] = 0
        got = F.flashopt_byte_product(a, b, F32)
        assert torch.equal(torch.diagonal(got)[1:16].cpu(), torch.tensor(want))


@pytest.mark.parametrize("m,n,k", [(1, 300, 4096), (20, 500, 1000), (300, 1100, 2200), (2100, 2100, 700),
                                   (4000, 3800, 300)])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_product_random(m, n, k, kind):
    """Any codes and scales."""
    require_gpu()
    a, b = _pair(m, n, k, 7 * m + n + k, kind, 100, 140, small=False)
    got = F.flashopt_byte_product(a, b, F32)
    _check_product(got, _values(a), _values(b))
    assert torch.equal(F.flashopt_byte_product(a, b), got.to(BF16))


def test_product_nan_scales():
    require_gpu()
    for m, n, k in ((3, 40, 300), (50, 700, 300), (300, 1100, 2200), (2100, 2100, 300)):
        a, b = _pair(m, n, k, 3)
        a.scales[1, 1], b.scales[n - 1, 0] = 255, 255
        got = F.flashopt_byte_product(a, b, F32)
        bad = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        bad[1], bad[:, n - 1] = True, True
        assert torch.equal(torch.isnan(got), bad)
        assert torch.equal(got[~bad].double(), (_values(a) @ _values(b).t())[~bad])


def test_product_last_scales():
    """Scale bytes at both ends: the sum of the two exponents is what counts."""
    require_gpu()
    for m, n, k in ((2, 30, 256), (300, 1100, 256)):
        a, b = _pair(m, n, k, 11)
        for sa, sb in ((0, 254), (254, 0), (0, 127), (127, 0), (254, 1), (1, 254), (64, 190)):
            a.scales[:, :2], b.scales[:, :2] = sa, sb
            assert torch.equal(F.flashopt_byte_product(a, b, F32).double(), _values(a) @ _values(b).t())


def test_product_views():
    """Outputs into views at any element; what lies around stays as it was."""
    require_gpu()
    for m, n, k in ((2, 33, 200), (50, 77, 200), (300, 1101, 300), (2100, 2101, 200), (4097, 4099, 130)):
        a, b = _pair(m, n, k, m)
        want = _values(a) @ _values(b).t()
        for dtype in (BF16, F32):
            for first in (0, 1, 3):
                wide = torch.full((m + 2, n + 7), 77.0, dtype=dtype, device="cuda")
                F.flashopt_byte_product(a, b, out=wide[1:m + 1, first:first + n])
                assert torch.equal(wide[1:m + 1, first:first + n], want.float().to(dtype))
                wide[1:m + 1, first:first + n] = 77
                assert (wide == 77).all()
    with pytest.raises(ValueError, match="columns"):
        F.flashopt_byte_product(a, _pair(3, 3, k + 1, 1)[1])
    with pytest.raises(ValueError, match="e4m3fn"):
        F.flashopt_byte_product(a, _pair(3, 3, k, 1, E5M2)[0])
    with pytest.raises(ValueError, match="overlap"):
        F.flashopt_byte_product(a, b, out=torch.zeros(n, device="cuda").expand(m, n))


# ------------------------------------------------------------------ linear

@pytest.mark.parametrize("m,k,n", [(1, 4096, 300), (1, 4095, 300), (2, 1000, 9000), (3, 136, 50), (4, 4096, 4096),
                                   (5, 4096, 700), (1, 14336, 4096), (4, 128, 20000), (48, 2000, 1000),
                                   (300, 1001, 1100), (1, 8, 5), (3, 2056, 16)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_is_quantize_and_product(m, k, n, dtype):
    require_gpu()
    x = _random(m, k, m + k, dtype, 3)
    w = F.flashopt_byte_quantize(_random(n, k, n, BF16, 2), block=True)
    for view in (x, torch.cat([x, x], 1)[:, 1:k + 1], x[:1].expand(m, k)):
        want = F.flashopt_byte_product(F.flashopt_byte_quantize(view), w, dtype)
        got = F.flashopt_byte_linear(view, w)
        assert got.dtype == dtype and torch.equal(got, want)
    wide = F.flashopt_byte_linear(x, w, F32)
    assert torch.equal(wide, F.flashopt_byte_product(F.flashopt_byte_quantize(x), w, F32))


def test_linear_non_finite():
    """A row with an infinity or NaN has NaN in every output, and no other row."""
    require_gpu()
    for m in (3, 40):
        x = _random(m, 1024, 4, BF16, 2)
        x[1, 1000], x[2, 3] = float("inf"), float("nan")
        w = F.flashopt_byte_quantize(_random(200, 1024, 5, BF16, 2))
        y = F.flashopt_byte_linear(x, w)
        assert torch.isnan(y[1:3]).all() and torch.isfinite(y[0]).all() and torch.isfinite(y[3:]).all()


def test_linear_workspace_and_out_between_columns():
    require_gpu()
    for m, k, n in ((1, 512, 100), (40, 512, 100), (300, 600, 1100)):
        both = torch.zeros(m, k + n + 3, dtype=BF16, device="cuda")
        both[:, :k] = _random(m, k, 1, BF16, 2)
        w = F.flashopt_byte_quantize(_random(n, k, 2, BF16, 2))
        want = F.flashopt_byte_linear(both[:, :k].contiguous(), w)
        work = torch.empty(F.flashopt_byte_linear_workspace_bytes(m, k), dtype=torch.uint8, device="cuda")
        F.flashopt_byte_linear(both[:, :k], w, out=both[:, k + 1:k + 1 + n], workspace=work)
        assert torch.equal(both[:, k + 1:k + 1 + n], want)
        with pytest.raises(F.FlashoptError, match="WORKSPACE"):
            F.flashopt_byte_linear(both[:, :k], w, workspace=work[:16])


# --------------------------------------------------------------- gradients

def _q(x, layout="rows", kind=E4M3, block=False):
    return _values(F.flashopt_byte_quantize(x.detach(), layout, block, kind))


@pytest.mark.parametrize("shape,n,dtype", [((1, 40), 30, BF16), ((33, 300), 129, BF16), ((2, 3, 100), 50, F32),
                                           ((1111, 1000), 777, BF16), ((300, 260), 1100, F32)])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("kind", [E4M3, E5M2])
def test_linear_gradients(shape, n, dtype, held, kind):
    """Against the formula in 64 bits, from the quantized operands."""
    require_gpu()
    k = shape[-1]
    x = _random(int(np.prod(shape[:-1])), k, n, dtype, 3).view(shape).requires_grad_()
    w = _random(n, k, n + 1, dtype, 2).requires_grad_()
    dy = _random(int(np.prod(shape[:-1])), n, n + 2, dtype, 4).view(*shape[:-1], n)
    weight = F.FP8Weight(w) if held else w
    y = F.fp8_linear(x, weight, grad_dtype=kind)
    assert y.shape == dy.shape and y.dtype == dtype
    y.backward(dy)
    fx, fdy = x.detach().view(-1, k), dy.view(-1, n)
    qw = _q(w, block=True)
    assert torch.equal(qw, _q(w, "cols", block=True).t())
    for got, a, b in ((y.view(-1, n), _q(fx), qw.t()), (x.grad.view(-1, k), _q(fdy, kind=kind), qw),
                      (w.grad, _q(fdy, "cols", kind), _q(fx, "cols").t())):
        _check_product(got, a, b.t())


def test_linear_gradient_against_differences():
    """Where the quantizers are exact (small integers, one scale), the layer is
    the linear one and a unit step of any operand moves the loss by its
    gradient, exactly."""
    require_gpu()
    g = torch.Generator().manual_seed(2)
    x = torch.randint(-8, 9, (70, 130), generator=g).to(BF16).cuda().requires_grad_()
    w = torch.randint(-8, 9, (40, 130), generator=g).to(BF16).cuda().requires_grad_()
    dy = torch.randint(-8, 9, (70, 40), generator=g).to(BF16).cuda()
    for t in (x, w, dy):
        t.data[:, ::128] = 8          # every group has one, along rows
        t.data[::128] = 8             # and along columns

    def loss(a, b):
        return float((F.flashopt_byte_product(F.flashopt_byte_quantize(a), F.flashopt_byte_quantize(b), F32).double()
                      * dy.double()).sum())
    F.fp8_linear(x, w).backward(dy)
    for t in (x, w):
        for i, j in ((1, 1), (5, 129), (39, 60)):
            with torch.no_grad():
                old, step = t[i, j].clone(), -1.0 if float(t[i, j]) > 0 else 1.0
                t[i, j] += step
                up = loss(x, w)
                t[i, j] = old
                assert (up - loss(x, w)) / step == float(t.grad[i, j].double()) or \
                    abs(float(t.grad[i, j]) - (up - loss(x, w)) / step) <= abs(float(t.grad[i, j])) * 2.0 ** -8


def test_weight_refresh():
    """An FP8Weight follows its parameter at refresh(); a backward pass that
    reads the copies of an older one refuses, one that does not runs."""
    require_gpu()
    x = _random(40, 256, 1, BF16, 2)
    w = _random(64, 256, 2, BF16, 2).requires_grad_()
    held = F.FP8Weight(w)
    codes = held.rows.codes.data_ptr()
    with torch.no_grad():
        w.mul_(3.0)
    assert torch.equal(F.fp8_linear(x, held), F.flashopt_byte_linear(x, F.flashopt_byte_quantize(w.detach() / 3, block=True)))
    held.refresh()
    assert held.rows.codes.data_ptr() == codes
    assert torch.equal(F.fp8_linear(x, held), F.fp8_linear(x, w))
    xg = x.clone().requires_grad_()
    y = F.fp8_linear(xg, held)
    held.refresh()
    with pytest.raises(RuntimeError, match="FP8Weight was refreshed"):
        y.sum().backward()
    y = F.fp8_linear(x, held)            # only the weight's gradient
    held.refresh()
    y.sum().backward()
    # written behind its back: autograd sees the new version
    y = F.fp8_linear(xg, held)
    F.flashopt_byte_quantize(w.detach(), "both", block=True, out=(held.rows, held.cols))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_captured_training_step():
    """Forward, backward, norm, clipped step and requantization in one graph;
    replays with new inputs, eager steps of a second copy between them, equal
    bits.  The captured parameter is in no eager graph."""
    require_gpu()
    rows, cols = 130, 200
    pa, pb = [W.init_param(rows * cols, device="cuda", seed=3).view(rows, cols).requires_grad_() for _ in range(2)]
    a, b = [F.FlashAdamW([p.detach()], **W.HP_DEFAULT) for p in (pa, pb)]
    wa, wb = F.FP8Weight(pa), F.FP8Weight(pb)
    x, dy = torch.zeros(70, cols, dtype=BF16, device="cuda"), torch.zeros(70, rows, dtype=BF16, device="cuda")
    grad, out = torch.zeros(rows, cols, dtype=BF16, device="cuda"), torch.zeros(2, device="cuda")
    norm, plan = F.GradPlan([grad]), a.plan([grad], step=1, grad_scale=out[1:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = F.fp8_linear(x, wa, grad_dtype=E5M2)
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
        z = F.fp8_linear(x, wb, grad_dtype=E5M2)
        z.backward(dy)
        eager = b.step([pb.grad], max_norm=0.01)
        pb.grad = None
        wb.refresh()
        torch.cuda.synchronize()
        assert torch.equal(y, z) and torch.equal(out, eager) and float(out[1]) < 1.0, t
        assert torch.equal(pa, pb) and torch.equal(a.states[0].block, b.states[0].block), t
        for q, r in ((wa.rows, wb.rows), (wa.cols, wb.cols)):
            assert torch.equal(q._buffer, r._buffer), t


def test_replayed_refresh_leaves_eager_passes_alone():
    """After a captured refresh, an eager forward pass keeps its own transposed
    copy: a replay before its backward pass does not reach it."""
    require_gpu()
    w = _random(64, 256, 2, BF16, 2).requires_grad_()
    held = F.FP8Weight(w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.refresh()
    graph.replay()
    x, dy = _random(40, 256, 1, BF16, 2).requires_grad_(), _random(40, 64, 3, BF16, 2)
    want, = torch.autograd.grad(F.fp8_linear(x, w), x, dy)
    y = F.fp8_linear(x, held)
    with torch.no_grad():
        w.mul_(-2.0)
    graph.replay()
    got, = torch.autograd.grad(y, x, dy)
    assert torch.equal(got, want)
    assert torch.equal(F.fp8_linear(x, held), F.fp8_linear(x, w))


# ------------------------------------------------------- streams and sizes

def test_other_stream():
    require_gpu()
    side = torch.cuda.Stream()
    x, w = _random(300, 700, 1, BF16, 2), _random(500, 700, 2, BF16, 2)
    want = F.flashopt_byte_linear(x, F.flashopt_byte_quantize(w, block=True))
    torch.cuda.synchronize()
    q = F.flashopt_byte_quantize(w, block=True, stream=side)
    got = F.flashopt_byte_linear(x, q, stream=side)
    rows = F.flashopt_byte_quantize(x, stream=side)
    again = F.flashopt_byte_product(rows, q, stream=side)
    values = F.flashopt_byte_dequantize(rows, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(again, want)
    assert torch.equal(values.double(), _values(rows))


def test_offsets_past_32_bits():
    """Codes of more than 4 GB: the last rows are those of the last rows alone.
    Integers of at most 8, so that their products are exact in any order."""
    require_gpu()
    rows, cols, last = 36000, 131072, 300
    g = torch.Generator().manual_seed(1)
    x = torch.empty(rows, cols, dtype=BF16, device="cuda")
    x.copy_(torch.arange(cols, device="cuda").remainder(251).to(BF16))
    x[-last:] = torch.randint(-8, 9, (last, cols), generator=g).to(BF16).cuda()
    q = F.flashopt_byte_quantize(x)
    tail = F.flashopt_byte_quantize(x[-last:])
    assert torch.equal(q.codes[-last:].view(torch.uint8), tail.codes.view(torch.uint8))
    assert torch.equal(q.scales[-last:], tail.scales)
    for m in (3, 300):
        a = torch.randint(-8, 9, (m, cols), generator=g).to(BF16).cuda()
        want = a.double() @ x[-last:].double().t()
        b = F.flashopt_byte_quantize(a)
        assert torch.equal(F.flashopt_byte_product(b, q, F32)[:, -last:].double(), want)
        assert torch.equal(F.flashopt_byte_product(q, b, F32)[-last:].t().double(), want)
    del q, tail
    t = F.flashopt_byte_quantize(x, "cols")
    end = F.flashopt_byte_quantize(x[:, -last:], "cols")
    assert torch.equal(t.codes[-last:].view(torch.uint8), end.codes.view(torch.uint8))
    assert torch.equal(t.scales[-last:], end.scales)
    v = F.flashopt_byte_dequantize(t, BF16)
    assert torch.equal(v[-last:], F.flashopt_byte_dequantize(end, BF16))
