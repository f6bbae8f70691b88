"""The library's 8-bit floating point operators as measured work: the codec of
E4M3 / E5M2 matrices with a power of two scale for each 128 elements, their
product and linear layer, and the root-mean-square norm with the residual's
addition in front of them, with gradients.

``run`` computes each in its plain form (elementary torch operations, 32 bits
or more) or, where ``own`` is true, through the library's entry points.
"""
import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64
E4M3, E5M2 = torch.float8_e4m3fn, torch.float8_e5m2
EPS = 1e-5


def _library():
    from bit_companded_adam_amd import flashopt
    return flashopt


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token through the norm and the 8.0B list's gate projection: the
        # residual's addition, the norm to 8 bits, the product with weights
        # laid out once
        dict(name="serve_token", op="serve", rows=1, inner=4096, outer=14336, residual=True),
        # a prompt through the same
        dict(name="serve_prompt", op="serve", rows=8192, inner=4096, outer=14336, residual=True),
        # one token, and a batch of decoding sequences, through the down
        # projection: an activation that comes in bf16, quantized on the way
        dict(name="linear_token", op="linear", rows=1, inner=14336, outer=4096),
        dict(name="linear_batch", op="linear", rows=48, inner=14336, outer=4096),
        # the norm's 8-bit output alone, for several products to share
        dict(name="norm8_prompt", op="norm8", rows=8192, cols=4096, both=False, fp32=False, residual=True),
        # a training activation, along tokens and along features, of an odd
        # fp32 matrix
        dict(name="norm8_odd", op="norm8", rows=333, cols=1001, both=True, fp32=True, residual=True),
        # the norm of the 1.2B list, forward and backward
        dict(name="norm_train_1b", op="norm", rows=8192, cols=2048, fp32=False, residual=True),
        dict(name="norm_train_odd", op="norm", rows=1111, cols=1001, fp32=True, residual=True),
        # the 8.0B list's gate weight after a step: one scale for each 128 x
        # 128 block, laid out for the forward and the backward product
        dict(name="codec_weight", op="codec", rows=14336, cols=4096, block=True, fp32=False, wide=False),
        # an odd output gradient with the wider exponent, along both axes
        dict(name="codec_odd", op="codec", rows=333, cols=1001, block=False, fp32=True, wide=True),
        # norm and linear layer of the 1.2B list, forward and backward
        dict(name="train_gate_1b", op="train", rows=8192, inner=2048, outer=5632, norm=True, wide=False),
        # an odd linear layer alone, gradients with the wider exponent
        dict(name="train_odd", op="train", rows=1111, inner=1000, outer=777, norm=False, wide=True),
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["serve", "linear", "norm8", "norm", "codec", "train"])
    rows = _log(rng, 1, 8192)

    def flag():
        return rng.random() < 0.5
    if op == "serve":
        return dict(op=op, rows=rows, inner=_log(rng, 33, 4096), outer=_log(rng, 33, 14336), residual=flag())
    if op == "linear":
        return dict(op=op, rows=min(rows, 2048), inner=_log(rng, 33, 14336), outer=_log(rng, 33, 4096))
    if op == "norm8":
        return dict(op=op, rows=rows, cols=_log(rng, 33, 4096), both=flag(), fp32=flag(), residual=flag())
    if op == "norm":
        return dict(op=op, rows=rows, cols=_log(rng, 33, 4096), fp32=flag(), residual=flag())
    if op == "codec":
        return dict(op=op, rows=rows, cols=_log(rng, 33, 4096), block=flag(), fp32=flag(), wide=flag())
    return dict(op=op, rows=rows, inner=_log(rng, 33, 2048), outer=_log(rng, 33, 5632), norm=flag(), wide=flag())


def work(case):
    op, m = case["op"], case["rows"]
    if op in ("norm8", "norm", "codec"):
        n, b = m * case["cols"], 4 if case["fp32"] else 2
        codes = 1 + 1 / 128 + 2             # 8 bits, their scale, and the bf16 values read back
        if op == "codec":
            return {"bytes": n * (b + 2 * codes), "flops": 4 * n}
        ends = 3 if case["residual"] else 1                # x, residual and their sum
        if op == "norm8":
            return {"bytes": n * (ends * b + codes * (2 if case["both"] else 1)), "flops": 6 * n}
        # forward, then both output gradients and the sum in, the input's gradient out
        return {"bytes": n * b * (ends + 1 + (4 if case["residual"] else 3)), "flops": 16 * n}
    k, n = case["inner"], case["outer"]
    weight = n * k * (1 + 1 / 128)
    if op in ("serve", "linear"):
        ends = 3 if op == "serve" and case["residual"] else 1
        return {"bytes": 2 * m * k * ends + weight + 2 * m * n, "flops": 2 * m * k * n}
    return {"bytes": 4 * (m * k * (2 if case["norm"] else 1) + n * k + m * n), "flops": 6 * m * k * n}


# ------------------------------------------------------------------ inputs

def _normal(seed, k, shape, std, dtype):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + k)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _factor(seed, k, shape):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 500_009 + k)
    return torch.exp(torch.randn(shape, generator=g, device="cuda"))


def prepare(case, seed):
    op, m = case["op"], case["rows"]
    k = case["cols"] if "cols" in case else case["inner"]
    dtype = F32 if case.get("fp32") else BF16
    # activations: some features are much larger than the others
    x = (_normal(seed, 0, (m, k), 1.0, F32) * _factor(seed, 1, k)).to(dtype)
    state = dict(case, x=x, eps=EPS)
    if op == "codec":
        return state
    if op == "serve" or op == "norm8" or op == "norm" or case.get("norm"):
        state["gain"] = (1.0 + _normal(seed, 2, k, 0.1, F32)).to(dtype)
        # a residual stream is larger than what a layer adds to it
        state["residual"] = _normal(seed, 3, (m, k), 4.0, dtype) if case.get("residual", True) else None
    if op == "norm8":
        return state
    if op in ("serve", "linear"):       # weights laid out once, as a serving program keeps them
        w = _normal(seed, 4, (case["outer"], k), 0.02, BF16)
        return dict(state, **dict(zip(("codes", "scales"), _codes(w, E4M3, True))))
    if op == "train":
        state["w"] = _normal(seed, 4, (case["outer"], k), 0.02, BF16).requires_grad_()
        state["dy"] = _normal(seed, 5, (m, case["outer"]), 1e-4, BF16)
    else:
        state["dy"] = _normal(seed, 5, (m, k), 1e-4, dtype)
    if state.get("residual") is not None:
        state["dh"] = _normal(seed, 6, (m, k), 1e-4, dtype)
        state["residual"].requires_grad_()
    if "gain" in state:
        state["gain"].requires_grad_()
    x.requires_grad_()
    return state


# ------------------------------------------------------ the plain operators

def _blocks(x):
    """x padded with zeros to whole blocks, as [row blocks, 128, column blocks, 128]."""
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 128, 0, -x.shape[0] % 128))
    return x.view(x.shape[0] // 128, 128, x.shape[1] // 128, 128)


def _codes(x, dtype, block):
    """8-bit codes [rows, cols padded to 128] and E8M0 bytes [rows, groups
    padded to 16] of a matrix: a scale for each 128 elements along its rows, or
    for each block of 128 x 128, the smallest power of two under which the
    largest magnitude is in range."""
    rows = x.shape[0]
    g = _blocks(x.detach().to(F32))
    top = g.abs().amax((1, 3) if block else 3, keepdim=True)
    m, e = torch.frexp(top)
    e = (e - (9 if dtype == E4M3 else 16) + (m > 0.875)).clamp(min=-127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = g * ((127 - e) << 23).view(F32)                  # times 2^-e, exact
    codes = y.reshape(g.shape[0] * 128, -1)[:rows].to(dtype)
    bytes_ = (e + 127).to(torch.uint8).expand(g.shape[0], 128, g.shape[2], 1).reshape(g.shape[0] * 128, -1)[:rows]
    return codes, torch.nn.functional.pad(bytes_, (0, -bytes_.shape[1] % 16)).contiguous()


def _values(codes, scales, cols):
    """The fp32 values that codes stand for."""
    b = scales[:, :codes.shape[1] // 128].to(torch.int32)
    unit = torch.where(b == 0, torch.full_like(b, 0x400000), b << 23).view(F32)
    return (codes.to(F32).view(codes.shape[0], -1, 128) * unit[..., None]).view(codes.shape)[:, :cols]


def _fp8(x, dtype=E4M3, block=False):
    return _values(*_codes(x, dtype, block), x.shape[1])


def _norm(state):
    """(y in fp32, h in the input's type, 1 / root in fp32)."""
    x, residual = state["x"], state["residual"]
    h = x if residual is None else (x.to(F32) + residual.to(F32)).to(x.dtype)
    r = (1.0 / (h.to(F64).square().mean(1, keepdim=True) + state["eps"]).sqrt()).to(F32)
    return h.to(F32) * r * state["gain"].to(F32), h, r


def _norm_grads(state, h, r, dy):
    """(gradient of the sum, gradient of the gain) in fp32."""
    u, t = dy * state["gain"].to(F32), h.to(F32) * r
    dx = r * (u - t * (u * t).mean(1, keepdim=True, dtype=F64).to(F32))
    if "dh" in state:
        dx = dx + state["dh"].to(F32)
    return dx, (dy * t).sum(0, dtype=F64).to(F32)


def _plain(state):
    op, x = state["op"], state["x"]
    if op == "codec":
        dtype = E5M2 if state["wide"] else E4M3
        return _fp8(x, dtype, state["block"]).to(BF16), _fp8(x.t(), dtype, state["block"]).to(BF16)
    if op == "linear":
        return (_fp8(x) @ _values(state["codes"], state["scales"], x.shape[1]).t()).to(BF16)
    if op == "train" and not state["norm"]:
        y, h = x.detach().to(F32), None
    else:
        y, h, r = _norm(state)
    if op == "serve":
        return (_fp8(y) @ _values(state["codes"], state["scales"], x.shape[1]).t()).to(BF16), h
    if op == "norm8":
        return [_fp8(y).to(BF16)] + ([_fp8(y.t()).to(BF16)] if state["both"] else []) + [h]
    if op == "norm":
        dx, dgain = _norm_grads(state, h, r, state["dy"].to(F32))
        return y.to(x.dtype), h, dx.to(x.dtype), dgain.to(x.dtype)
    w, dy, kind = state["w"], state["dy"], E5M2 if state["wide"] else E4M3
    q = _fp8(w, E4M3, True)
    out = (_fp8(y) @ q.t()).to(BF16)
    dx = _fp8(dy, kind) @ q
    dw = (_fp8(dy.t(), kind) @ _fp8(y.t()).t()).to(BF16)
    if not state["norm"]:
        return out, dx.to(BF16), dw
    dx, dgain = _norm_grads(state, h, r, dx)
    return out, h, dx.to(BF16), dgain.to(BF16), dw


# ---------------------------------------------------- the library's operators

def _calls(state):
    F, op, x = _library(), state["op"], state["x"]
    if op == "codec":
        rows, cols = F.flashopt_byte_quantize(x, "both", block=state["block"], dtype=E5M2 if state["wide"] else E4M3)
        return F.flashopt_byte_dequantize(rows, BF16), F.flashopt_byte_dequantize(cols, BF16)
    if op in ("serve", "linear"):
        w = F.FP8Tensor(state["codes"], state["scales"], state["outer"], state["inner"])
        if op == "linear":
            return F.flashopt_byte_linear(x, w)
        q, h = F.flashopt_rms_norm(x, state["gain"], state["residual"], eps=state["eps"], output="rows")
        return F.flashopt_byte_product(q, w), h
    if op == "norm8":
        q, h = F.flashopt_rms_norm(x, state["gain"], state["residual"], eps=state["eps"],
                                   output="both" if state["both"] else "rows")
        return [F.flashopt_byte_dequantize(t, BF16) for t in (q if state["both"] else (q,))] + [h]
    # a layer without a residual has no gradient of the sum from elsewhere
    sides = ((state["dy"], state["dh"]) if "dh" in state else (state["dy"],))
    if op == "norm":
        y, h = F.rms_norm(x, state["gain"], state["residual"], eps=state["eps"])
        return (y, h, *torch.autograd.grad((y, h)[:len(sides)], (x, state["gain"]), sides))
    grad = E5M2 if state["wide"] else E4M3
    if not state["norm"]:
        y = F.fp8_linear(x, state["w"], grad_dtype=grad)
        return (y, *torch.autograd.grad(y, (x, state["w"]), sides))
    y, h = F.fp8_norm_linear(x, state["gain"], state["w"], state["residual"], eps=state["eps"], grad_dtype=grad)
    return (y, h, *torch.autograd.grad((y, h), (x, state["gain"], state["w"]), sides))


def run(state):
    if own:
        return _calls(state)
    with torch.no_grad():
        return _plain(state)


# ------------------------------------------------------- in 64 bits, apart

def _exact_fp8(x, bits=3, low=-6, top=448.0, axis=1, block=False):
    """Values of the 8-bit rounding in double: the unit doubles from 2^-127 on
    until the largest magnitude fits; a value's step is 2^-bits of its own
    binade, not below that of 2^low units."""
    x = x.to(F64)
    rows, cols = x.shape
    far = x.new_zeros(rows + -rows % 128, cols + -cols % 128)
    far[:rows, :cols] = x.abs()
    if block:
        largest = far.unflatten(0, (-1, 128)).unflatten(2, (-1, 128)).amax((1, 3))
        largest = largest.repeat_interleave(128, 0).repeat_interleave(128, 1)
    else:
        largest = far.unflatten(axis, (-1, 128)).amax(axis + 1).repeat_interleave(128, axis)
    largest = largest[:rows, :cols]
    # the exponent field of largest / top, rounded up to a power of two
    ratio = (largest / top).contiguous().view(torch.int64)
    whole = (ratio & ((1 << 52) - 1)) == 0
    power = torch.where(largest == 0, torch.full_like(ratio, -127), (ratio >> 52) - 1023 + (~whole).long())
    power = power.clamp(min=-127)
    unit = ((power + 1023) << 52).view(F64)
    y = x / unit
    binade = (((y.contiguous().view(torch.int64) >> 52) & 2047) - 1023).clamp(min=low)
    step = ((binade - bits + 1023) << 52).view(F64)
    return torch.round(y / step) * step * unit


def exact(case, seed):
    s = prepare(case, seed)
    op, x = case["op"], s["x"].detach().to(F64)
    e5m2 = dict(bits=2, low=-14, top=57344.0)
    grad = e5m2 if case.get("wide") else {}
    if op == "codec":
        return (_exact_fp8(x, block=case["block"], **grad),
                _exact_fp8(x, block=case["block"], axis=0, **grad).t())
    y, h = x, None
    if "gain" in s:
        # the sum is held in the input's type: that rounding is part of the operator
        h = x if s["residual"] is None else (x + s["residual"].detach().to(F64)).to(s["x"].dtype).to(F64)
        gain = s["gain"].detach().to(F64)
        root = torch.sqrt(h.pow(2).sum(1) / h.shape[1] + EPS)[:, None]
        unit = h / root
        y = unit * gain

    def norm_grads(dy):
        g = dy * gain / root
        dx = g - h * (g * h).sum(1, keepdim=True) / (root * root * h.shape[1])
        return dx + s["dh"].to(F64) if "dh" in s else dx, (dy * unit).sum(0)
    if op == "norm8":
        return [_exact_fp8(y)] + ([_exact_fp8(y, axis=0).t()] if case["both"] else []) + [h]
    if op == "norm":
        return (y, h, *norm_grads(s["dy"].to(F64)))
    if op in ("serve", "linear"):
        n, k = case["outer"], case["inner"]
        unit_w = torch.pow(torch.full((), 2.0, dtype=F64, device=x.device), s["scales"].to(F64) - 127)
        w = torch.zeros(n, k, dtype=F64, device=x.device)
        for first in range(0, k, 128):
            w[:, first:first + 128] = s["codes"][:, first:min(k, first + 128)].to(F64) * unit_w[:, first // 128, None]
        out = torch.matmul(_exact_fp8(y), w.t())
        return (out, h) if op == "serve" else out
    w, dy = _exact_fp8(s["w"].detach(), block=True), s["dy"].to(F64)
    out = _exact_fp8(y) @ w.t()
    dy_w = _exact_fp8(dy, **grad) @ w
    dw = _exact_fp8(dy, axis=0, **grad).t() @ _exact_fp8(y, axis=0)
    if not case["norm"]:
        return out, dy_w, dw
    return (out, h, *norm_grads(dy_w), dw)
