"""The library's training operators next to the fused step, as measured work:
the global gradient norm over a tensor list, clipping by it in place, the
clipped FlashAdamW step, and the microscaled 4-bit (MXFP4) codec, product and
linear layer.

``run`` computes each in its plain form (elementary torch operations, 32 bits
or more) or, where ``own`` is true, through the library's entry points.
"""
import torch

own = False

F32, BF16, F64 = torch.float32, torch.bfloat16, torch.float64


def _library():
    from bit_companded_adam_amd import flashopt
    return flashopt


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the gradients of the 1.2B decoder list, all bf16: the norm that a
        # training step logs and clips by
        dict(name="norm_decoder_1b", op="norm", vocab=32000, d=2048, kv=2048, f=5632, layers=22),
        # a short ragged list with fp32 gradients among the bf16 ones
        # (adapters, norm vectors, biases): latency counts
        dict(name="norm_ragged", op="norm", count=24, top=70001),
        # one layer of the 8.0B decoder list clipped in place, for an
        # optimizer that takes its gradients already clipped
        dict(name="clip_decoder_8b_layer", op="clip", vocab=0, d=4096, kv=1024, f=14336, layers=1),
        dict(name="clip_ragged", op="clip", count=40, top=70001),
        # the norm and the clipped fused step over one layer of the 8.0B list,
        # bf16 parameters with fp32 moments
        dict(name="step_decoder_8b_layer", op="step", vocab=0, d=4096, kv=1024, f=14336, layers=1,
             codes=False),
        # the same with the 24-bit master and companded moments on the single
        # 2^20 tensor of the benchmark, its state returned as values
        dict(name="step_codes_1m", op="step", count=1, top=1 << 20, codes=True),
        # an activation of 8192 tokens, quantized along tokens and along
        # features in one pass, and read back
        dict(name="codec_activation", op="codec", rows=8192, cols=4096, fp32=False),
        # an odd fp32 matrix: ragged groups in both directions
        dict(name="codec_odd", op="codec", rows=333, cols=1001, fp32=True),
        # one token, and a prompt, through the 8.0B list's gate projection
        dict(name="product_token", op="product", rows=1, inner=4096, outer=14336),
        dict(name="product_prompt", op="product", rows=8192, inner=4096, outer=14336),
        # a linear layer of the 1.2B list, forward and backward
        dict(name="train_gate_1b", op="train", rows=8192, inner=2048, outer=5632),
        dict(name="train_odd", op="train", rows=1111, inner=1000, outer=777),
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng):
    op = rng.choice(["norm", "clip", "step", "codec", "product", "train"])
    if op in ("norm", "clip", "step"):
        case = dict(op=op)
        if rng.random() < 0.5:
            case |= dict(count=rng.randint(1, 14 if op == "step" else 48), top=_log(rng, 33, 1 << 20))
        else:
            d = 64 * _log(rng, 4, 64 if op == "norm" else 32)
            case |= dict(vocab=_log(rng, 100, 16000), d=d, kv=max(64, d // rng.choice([1, 4])),
                         f=_log(rng, d, 3 * d), layers=rng.randint(1, 3 if op == "norm" else 1))
        if op == "step":
            case["codes"] = rng.random() < 0.5
        return case
    if op == "codec":
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 33, 4096), fp32=rng.random() < 0.5)
    rows = _log(rng, 1, 8192)
    if op == "product":
        return dict(op=op, rows=rows, inner=_log(rng, 33, 4096), outer=_log(rng, 33, 14336))
    return dict(op=op, rows=rows, inner=_log(rng, 33, 2048), outer=_log(rng, 33, 5632))


def _list(case):
    """(sizes, fp32 flags) of a gradient list: a decoder's tensors, or a
    ragged list whose sizes run evenly in their logarithm up to the top."""
    if "count" in case:
        n, top = case["count"], case["top"]
        sizes = [top if n == 1 else max(1, round(top ** (i / (n - 1)))) for i in range(n)]
        return sizes, [case["op"] != "step" and i % 3 == 2 for i in range(n)]
    d, kv, f = case["d"], case["kv"], case["f"]
    sizes = [case["vocab"] * d] if case["vocab"] else []
    sizes += [d * d, d * kv, d * kv, d * d, d * f, d * f, f * d, d, d] * case["layers"]
    return sizes, [False] * len(sizes)


def work(case):
    op = case["op"]
    if op in ("norm", "clip", "step"):
        sizes, wide = _list(case)
        n, b = sum(sizes), sum(s * (4 if w else 2) for s, w in zip(sizes, wide))
        if op == "norm":
            return {"bytes": b + 8, "flops": 2 * n}
        if op == "clip":
            return {"bytes": 2 * b + 8, "flops": 3 * n}
        # gradient and parameter, then fp32 moments both ways, or codes with
        # their scales and corrections both ways and three fp32 values out
        return {"bytes": n * (12.25 + 12 if case["codes"] else 22) + 8, "flops": 16 * n}
    if op == "codec":
        n = case["rows"] * case["cols"]
        return {"bytes": n * ((4 if case["fp32"] else 2) + 2 * 17 / 32 + 4), "flops": 4 * n}
    m, k, n = case["rows"], case["inner"], case["outer"]
    if op == "product":
        return {"bytes": 2 * m * k + 17 / 32 * n * k + 2 * m * n, "flops": 2 * m * k * n}
    return {"bytes": 4 * (m * k + n * k + m * n), "flops": 6 * m * k * n}


# ------------------------------------------------------------------ inputs

def _normal(seed, k, shape, std, dtype):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + k)
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _factor(seed, k, shape):
    g = torch.Generator(device="cuda").manual_seed(1_000_003 * seed + 500_009 + k)
    return torch.exp(torch.randn(shape, generator=g, device="cuda"))


HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01)


def prepare(case, seed):
    op = case["op"]
    if op in ("norm", "clip", "step"):
        sizes, wide = _list(case)
        # N(0, 1e-3) times a lognormal factor for each tensor
        factor = _factor(seed, 0, len(sizes)).tolist()
        grads = [_normal(seed, i, n, 1e-3 * f, F32 if w else BF16)
                 for i, (n, w, f) in enumerate(zip(sizes, wide, factor))]
        state = dict(case, grads=grads, max_norm=0.25 * 1e-3 * sum(sizes) ** 0.5)
        if op == "step":
            state["params"] = [_normal(seed, 10_000 + i, n, 0.02, BF16) for i, n in enumerate(sizes)]
        return state
    if op == "codec":
        # an activation: some features are much larger than the others
        x = _normal(seed, 0, (case["rows"], case["cols"]), 1.0, F32) * _factor(seed, 1, case["cols"])
        return dict(case, x=x if case["fp32"] else x.to(BF16))
    m, k, n = case["rows"], case["inner"], case["outer"]
    x = (_normal(seed, 0, (m, k), 1.0, F32) * _factor(seed, 1, k)).to(BF16)
    w = _normal(seed, 2, (n, k), 0.02, BF16)
    if op == "product":      # weights laid out once, as a serving program keeps them
        codes, scales = _pack(*_mx_codes(w))
        return dict(case, x=x, codes=codes, scales=scales)
    dy = _normal(seed, 3, (m, n), 1e-4, BF16)
    return dict(case, x=x.requires_grad_(), w=w.requires_grad_(), dy=dy)


# ------------------------------------------------------ the plain operators

def _norm_and_scale(grads, max_norm):
    total = torch.stack([g.to(F32).square().sum(dtype=F64) for g in grads]).sum()
    norm = total.sqrt()
    scale = (max_norm / (norm + 1e-6)).clamp(max=1.0)
    return torch.stack([norm, scale]).to(F32)


def _clip(grads, max_norm):
    out = _norm_and_scale(grads, max_norm)
    return out, [g.copy_(g.to(F32) * out[1]) for g in grads]


def _groups(x):
    """The groups of 32 of a flat tensor, the last one padded with zeros."""
    return torch.cat([x, x.new_zeros(-x.numel() % 32)]).view(-1, 32)


def _companded(a, levels, signed):
    """Group-32 codes of a under its fp16 scale: (code / levels, scale)."""
    g = _groups(a)
    s = (g.abs() if signed else g).amax(1, keepdim=True).to(torch.float16).to(F32)
    y = g / torch.where(s == 0, torch.ones_like(s), s)
    y = 2.0 * y / (1.0 + y.abs()) if signed else y
    # divided by a tensor: dividing by a number multiplies by its reciprocal
    q = torch.round(y * levels).clamp(-levels if signed else 0, levels) / torch.full_like(s, levels)
    return q, s


def _momentum(m):
    q, s = _companded(m, 127.0, True)
    return (q / (2.0 - q.abs()) * s).view(-1)[:m.numel()]


def _variance(v):
    q, s = _companded(v.sqrt(), 255.0, False)
    return (q * s).square().view(-1)[:v.numel()]


def _split(theta):
    """The bf16 parameter (nearest, ties away from zero) and the value of the
    24-bit master: the correction in 1/256 of a bf16 step, half to even."""
    bits = theta.view(torch.int32)
    top = (bits + 0x8000) & -0x10000
    rho = torch.round((bits - top).to(F32) / 256.0).clamp(-128, 127).to(torch.int32)
    return top.view(F32).to(BF16), (top + rho * 256).view(F32)


def _adamw(p, master, m, v, g, t, codes):
    """One tensor's step in place, one fp32 rounding for each operation."""
    b1, b2 = HYPER["betas"]
    theta = master * (1.0 - HYPER["lr"] * HYPER["weight_decay"])
    m1 = b1 * m + (1.0 - b1) * g
    v1 = b2 * v + (1.0 - b2) * g * g
    # the bias corrections as fp32 tensors: an elementwise quotient
    c1, c2 = torch.full_like(m1[:1], 1.0 - b1 ** t), torch.full_like(m1[:1], 1.0 - b2 ** t)
    theta = theta - HYPER["lr"] * (m1 / c1) / ((v1 / c2).sqrt() + HYPER["eps"])
    if not codes:
        p.copy_(theta)
        return p, m.copy_(m1), v.copy_(v1)
    param, value = _split(theta)
    return p.copy_(param), m.copy_(_momentum(m1)), v.copy_(_variance(v1)), master.copy_(value)


def _clipped_step(state):
    params, codes = state["params"], state["codes"]
    if "t" not in state:
        state["t"] = 0
        state["m"] = [torch.zeros_like(p, dtype=F32) for p in params]
        state["v"] = [torch.zeros_like(p, dtype=F32) for p in params]
        state["master"] = [p.to(F32) for p in params] if codes else None
    state["t"] += 1
    out = _norm_and_scale(state["grads"], state["max_norm"])
    masters = state["master"] or [p.to(F32) for p in params]
    return out, [_adamw(p, w, m, v, g.to(F32) * out[1], state["t"], codes)
                 for p, w, m, v, g in zip(params, masters, state["m"], state["v"], state["grads"])]


GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_codes(x):
    """MXFP4 codes [rows, cols padded to 128] and E8M0 bytes [rows, groups]
    of a matrix, groups of 32 along its rows."""
    x = x.detach().to(F32)
    x = torch.nn.functional.pad(x, (0, -x.shape[1] % 128))
    g = x.reshape(x.shape[0], -1, 32)
    top = g.abs().amax(2)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = g * ((127 - e) << 23).view(F32)[..., None]       # times 2^-e, exact
    a = y.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    return (code | (torch.signbit(y).to(torch.uint8) << 3)).view(x.shape), (e + 127).to(torch.uint8)


def _pack(codes, scales):
    return codes[:, 0::2] | (codes[:, 1::2] << 4), scales


def _mx_values(codes, scales, cols):
    """The fp32 values that unpacked codes stand for."""
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    b = scales.to(torch.int32)
    unit = torch.where(b == 0, torch.full_like(b, 0x400000), b << 23).view(F32)
    v = grid[codes.to(torch.int32)].view(codes.shape[0], -1, 32) * unit[..., None]
    return v.reshape(codes.shape)[:, :cols]


def _mx(x):
    return _mx_values(*_mx_codes(x), x.shape[1])


def _plain(state):
    op = state["op"]
    if op == "norm":
        return _norm_and_scale(state["grads"], state["max_norm"])
    if op == "clip":
        return _clip(state["grads"], state["max_norm"])
    if op == "step":
        return _clipped_step(state)
    x = state["x"]
    if op == "codec":
        return _mx(x).to(BF16), _mx(x.t()).to(BF16)
    if op == "product":
        packed = state["codes"]
        codes = torch.stack([packed & 15, packed >> 4], 2).view(packed.shape[0], -1)
        return (_mx(x) @ _mx_values(codes, state["scales"], x.shape[1]).t()).to(BF16)
    w, dy = state["w"], state["dy"]
    y = _mx(x) @ _mx(w).t()
    dx = _mx(dy) @ _mx(w.t()).t()
    dw = _mx(dy.t()) @ _mx(x.t()).t()
    return y.to(BF16), dx.to(BF16), dw.to(BF16)


# ---------------------------------------------------- the library's operators

def _step_calls(F, state):
    if "opt" not in state:
        codes = state["codes"]
        state["opt"] = F.FlashAdamW(state["params"], master_bits=24 if codes else None,
                                    quantize_states=codes, state_layout="streams", **HYPER)
    opt = state["opt"]
    out = opt.step(state["grads"], max_norm=state["max_norm"])
    if not state["codes"]:
        return out, [(s.param, s.m_codes, s.v_codes) for s in opt.states]
    return out, [(s.param, F.flashopt_dequantize(s.m_codes, s.m_scales, F.SPEC_MOMENTUM),
                  F.flashopt_dequantize(s.v_codes, s.v_scales, F.SPEC_VARIANCE),
                  F.flashopt_reconstruct(s.param, s.rho, 24)) for s in opt.states]


def _calls(state):
    F, op = _library(), state["op"]
    if op == "norm":
        return F.flashopt_grad_norm(state["grads"], state["max_norm"])
    if op == "clip":
        return F.flashopt_grad_clip(state["grads"], state["max_norm"]), state["grads"]
    if op == "step":
        return _step_calls(F, state)
    x = state["x"]
    if op == "codec":
        rows, cols = F.flashopt_mx_quantize(x, layout="both")
        return F.flashopt_mx_dequantize(rows, BF16), F.flashopt_mx_dequantize(cols, BF16)
    if op == "product":
        w = F.MXTensor(state["codes"], state["scales"], state["outer"], state["inner"])
        return F.flashopt_mx_linear(x, w)
    y = F.mx_linear(x, state["w"])
    return (y, *torch.autograd.grad(y, (x, state["w"]), state["dy"]))


def run(state):
    if state["op"] == "clip":
        # gradients clipped in place stay clipped, so each pass asks for a
        # little less than the last: every pass has values to scale
        state["max_norm"] *= 0.999
    if own:
        return _calls(state)
    with torch.no_grad():
        return _plain(state)


# ------------------------------------------------------- in 64 bits, apart

def _two_to(e):
    """2^e in double by its bits (a power of a tensor may be an ulp off)."""
    return ((e.to(torch.int64) + 1023) << 52).view(F64)


def _exact_mx(x, axis):
    """Values of the MXFP4 rounding in double: within a group, the step is a
    power of two below the value's own, and at least half the group's unit."""
    x = x.detach().to(F64).movedim(axis, -1)
    n = x.shape[-1]
    g = torch.nn.functional.pad(x, (0, -n % 32)).unflatten(-1, (-1, 32))
    top = g.abs().amax(-1, keepdim=True)
    unit = _two_to((torch.frexp(top)[1] - 3).clamp(min=-127))
    y = g / unit
    step = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
    v = (torch.round(y / step) * step).clamp(-6, 6) * unit
    return v.flatten(-2)[..., :n].movedim(-1, axis)


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "clip", "step"):
        grads = state["grads"]
        if op == "clip":
            state["max_norm"] *= 0.999
        norm = sum(float(torch.dot(g.to(F64), g.to(F64))) for g in grads) ** 0.5
        scale = min(1.0, state["max_norm"] / (norm + 1e-6))
        out = torch.tensor([norm, scale], dtype=F64)
        if op == "norm":
            return out
        if op == "clip":
            return out, [g.to(F64) * scale for g in grads]
        done = []
        for p, g in zip(state["params"], grads):     # the first step, from empty moments
            g, p = g.to(F64) * scale, p.to(F64)
            m, v = (1 - 0.9) * g, (1 - 0.999) * g ** 2
            root = (v / (1 - 0.999)).sqrt() + HYPER["eps"]
            theta = p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - HYPER["lr"] * (m / (1 - 0.9)) / root
            # values of codes and corrections follow fp32 roundings: no 64-bit value
            done.append((theta, None, None, None) if case["codes"] else (theta, m, v))
        return out, done
    x = state["x"]
    if op == "codec":
        return _exact_mx(x, 1), _exact_mx(x, 0).t()
    if op == "product":
        signed = [float((1 - 2 * (c >> 3)) * GRID[c & 7]) for c in range(16)]
        table = torch.tensor(signed, dtype=F64, device=x.device)
        n, k = case["outer"], case["inner"]
        nibbles = torch.empty(n, 2 * state["codes"].shape[1], dtype=F64, device=x.device)
        nibbles[:, 0::2] = table[(state["codes"] % 16).long()]
        nibbles[:, 1::2] = table[torch.div(state["codes"], 16, rounding_mode="floor").long()]
        unit = _two_to(state["scales"].to(torch.int32) - 127)
        w = (nibbles.view(n, -1, 32) * unit[:, :, None]).view(n, -1)[:, :k]
        return torch.matmul(_exact_mx(x, 1), w.t())
    w, dy = state["w"], state["dy"]
    return (_exact_mx(x, 1) @ _exact_mx(w, 1).t(), _exact_mx(dy, 1) @ _exact_mx(w, 0),
            _exact_mx(dy, 0).t() @ _exact_mx(x, 0))
