"""Microscaled storage and the linear layer on it: cases, their plain form, and the library's calls.

Values are held in blocks of 32 along a row: 4-bit (E2M1, ``fp4``) or 8-bit
(E4M3, ``fp8``) floating-point codes, and one power of two a block (a byte b
for 2^(b - 127)).  Three operators:

* ``save`` and ``payload``: quantisation of a matrix (an activation kept for
  the backward pass, the parameters' copy for a 4-bit all-gather), the second
  with the dequantisation that a receiver makes of it;
* ``linear`` and ``product``: y = x w^T with w in blocks, x in bf16 or in
  blocks itself;
* ``dgrad`` and ``wgrad``: its backward, dx = dy w and dw = dy^T x, the latter
  from the activation kept in blocks.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, with the calls a user makes of sharded_mixed_precision_shard_amd.
"""
import functools
import math

import torch

own = False

BLOCK = 32
WORKSPACE = 1 << 26   # bytes that a program keeps for the products
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
# largest exponent, smallest exponent, bits of mantissa, largest value
FORMS = {"fp4": (2, 0, 1, 6.0), "fp8": (8, -6, 3, 448.0)}


def listed():
    return [
        # a small activation of odd sizes in fp32: nothing but latency
        dict(name="save, small odd", op="save", form="fp8", type="fp32", rows=37, cols=1001, pad=3),
        # the input of a 7B model's layer, 16384 tokens, kept for the backward pass
        dict(name="save, 7B layer", op="save", form="fp8", type="bf16", rows=16384, cols=4096,
             pad=0),
        # a 7B model's shard on 8 ranks: the 4-bit copy for the all-gather, and reading it back
        dict(name="payload, 7B shard", op="payload", form="fp4", type="bf16", rows=1,
             cols=805388288, pad=0),
        # one token through a 7B model's first MLP matrix: bound by the weights' bytes
        dict(name="linear, one token", op="linear", w="fp4", m=1, n=11008, k=4096, pad=0),
        # a ragged batch of odd sizes, rows of x apart by an odd stride
        dict(name="linear, ragged batch", op="linear", w="fp4", m=37, n=1003, k=4101, pad=3),
        # a training batch through a 7B model's first MLP matrix
        dict(name="linear, 7B layer", op="linear", w="fp4", m=8192, n=11008, k=4096, pad=0),
        # eight sequences' next tokens through a 70B model's MLP matrix, both sides in blocks
        dict(name="product, few tokens", op="product", x="fp4", w="fp4", m=8, n=28672, k=8192),
        # a long batch through the same matrix
        dict(name="product, 70B layer", op="product", x="fp4", w="fp4", m=8192, n=28672, k=8192),
        # a small layer's input gradient, odd sizes
        dict(name="dgrad, odd", op="dgrad", w="fp4", m=515, n=1003, k=770, pad=1),
        # the input gradient of a 7B model's first MLP matrix
        dict(name="dgrad, 7B layer", op="dgrad", w="fp4", m=8192, n=11008, k=4096, pad=0),
        # a small model's square matrix over a long batch, added to fp32 gradients
        dict(name="wgrad, small layer", op="wgrad", x="fp8", m=16384, n=768, k=768, pad=0,
             type="fp32", add=True),
        # the partial of a 7B model's second MLP matrix
        dict(name="wgrad, 7B layer", op="wgrad", x="fp8", m=8192, n=4096, k=11008, pad=0,
             type="bf16", add=False),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("save", "payload", "linear", "linear", "product", "dgrad", "wgrad"))
    pad = rng.choice((0, 0, 8, 1))
    if op in ("save", "payload"):
        cols = _between(rng, 1, 16384)
        rows = _between(rng, 1, max(1, 134217728 // cols))
        return dict(op=op, form=rng.choice(("fp8", "fp4")) if op == "payload" else "fp8",
                    type=rng.choice(tuple(TYPES)), rows=rows, cols=cols, pad=pad)
    m, n, k = (_between(rng, 1, 8192), _between(rng, 16, 16384), _between(rng, 16, 14000))
    if rng.random() < 0.6:  # most layers' widths are round, batches are not
        n, k = -(-n // 64) * 64, -(-k // 64) * 64
    if op == "linear":
        return dict(op=op, w=rng.choice(("fp4", "fp4", "fp8")), m=m, n=n, k=k, pad=pad)
    if op == "product":
        return dict(op=op, x=rng.choice(("fp4", "fp8")), w="fp4", m=m, n=n, k=k)
    if op == "dgrad":
        return dict(op=op, w="fp4", m=m, n=n, k=k, pad=pad)
    kind = rng.choice(("bf16", "fp32"))
    return dict(op=op, x="fp8", m=m, n=n, k=k, pad=pad, type=kind,
                add=kind == "fp32" and rng.random() < 0.5)


def _width(form, cols):
    """Bytes of a row's codes: whole blocks."""
    return -(-cols // BLOCK) * BLOCK * (4 if form == "fp4" else 8) // 8


def _matrix(rows, cols, pad, dtype, gen, sigma, outliers=False):
    """A normal matrix whose rows lie cols + pad elements apart; activations have a few
    channels of large values."""
    x = torch.empty((rows, cols + pad), dtype=dtype, device=gen.device)
    x.normal_(0.0, sigma, generator=gen)
    if outliers:
        x[:, 17::128] *= 12.0
    return x[:, :cols]


def prepare(case, seed):
    gen = torch.Generator(device=torch.device("cuda", torch.cuda.current_device()))
    gen.manual_seed(seed)
    s = dict(case)
    op, device = case["op"], gen.device

    def blocks(form, rows, cols, sigma, outliers=False):
        x = _matrix(rows, cols, 0, torch.bfloat16, gen, sigma, outliers)
        return _quantise(x, form)

    if op in ("save", "payload"):
        rows, cols = case["rows"], case["cols"]
        sigma = 1.0 if op == "save" else 0.02
        s["in"] = _matrix(rows, cols, case["pad"], TYPES[case["type"]], gen, sigma, op == "save")
        s["codes"] = torch.zeros((rows, _width(case["form"], cols)), dtype=torch.uint8,
                                 device=device)
        s["scales"] = torch.zeros((rows, -(-cols // BLOCK)), dtype=torch.uint8, device=device)
        if op == "payload":
            s["out"] = torch.zeros((rows, cols), dtype=TYPES[case["type"]], device=device)
        return s
    m, n, k = case["m"], case["n"], case["k"]
    s["workspace"] = torch.zeros(WORKSPACE, dtype=torch.uint8, device=device)
    if op == "linear":
        s["in"] = _matrix(m, k, case["pad"], torch.bfloat16, gen, 1.0, True)
        s["codes"], s["scales"] = blocks(case["w"], n, k, 0.02)
        s["out"] = torch.zeros((m, n), dtype=torch.bfloat16, device=device)
    elif op == "product":
        s["xcodes"], s["xscales"] = blocks(case["x"], m, k, 1.0, True)
        s["codes"], s["scales"] = blocks(case["w"], n, k, 0.02)
        s["out"] = torch.zeros((m, n), dtype=torch.bfloat16, device=device)
    elif op == "dgrad":
        s["in"] = _matrix(m, n, case["pad"], torch.bfloat16, gen, 1e-3)
        s["codes"], s["scales"] = blocks(case["w"], n, k, 0.02)
        s["out"] = torch.zeros((m, k), dtype=torch.bfloat16, device=device)
    else:
        s["in"] = _matrix(m, n, case["pad"], torch.bfloat16, gen, 1e-3)
        s["codes"], s["scales"] = blocks(case["x"], m, k, 1.0, True)
        s["out"] = torch.empty((n, k), dtype=TYPES[case["type"]], device=device)
        s["out"].normal_(0.0, 1e-2, generator=gen)
    return s


def _quantise(x, form):
    """Codes and scales of a matrix, rows padded with zeros to whole blocks."""
    top, low, bits, most = FORMS[form]
    rows, cols = x.shape
    count = -(-cols // BLOCK)
    v = torch.nn.functional.pad(x.float(), (0, count * BLOCK - cols)).view(rows, count, BLOCK)
    peak = v.abs().amax(2, keepdim=True)
    good = torch.isfinite(peak)
    e = torch.frexp(peak)[1].int().sub_(1 + top).clamp_(-127, 127)
    e = torch.where(peak > 0, e, torch.full_like(e, -127))
    v = torch.where(good, torch.ldexp(v, -e), torch.zeros_like(v))
    scales = torch.where(good, e + 127, torch.full_like(e, 255)).to(torch.uint8).view(rows, count)
    size = v.abs()
    step = torch.frexp(size)[1].int().sub_(1).clamp_(low, top).sub_(bits)
    whole = torch.round(torch.ldexp(size, -step))  # to even
    size = torch.ldexp(whole, step).clamp_(max=most)
    # code: exponent field and mantissa of the rounded value
    field = torch.frexp(size)[1].int().sub_(1).clamp_(low, top)
    field = torch.where(size > 0, field, torch.full_like(field, low))
    mantissa = torch.ldexp(size, bits - field).int()
    code = ((field - low) << bits) + mantissa
    code += torch.signbit(v).int() << (3 if form == "fp4" else 7)
    code = code.to(torch.uint8).view(rows, count * BLOCK)
    if form == "fp4":
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    return code.contiguous(), scales


@functools.lru_cache(maxsize=None)
def _table(form, device):
    """The value of every code."""
    top, low, bits, most = FORMS[form]
    code = torch.arange(16 if form == "fp4" else 256, device=device)
    half = code.numel() // 2
    mantissa, field = (code % half) & ((1 << bits) - 1), (code % half) >> bits
    power = (field - 1).clamp(min=0) + (low - bits)
    value = torch.ldexp((mantissa + (field > 0).int() * (1 << bits)).float(), power)
    if form == "fp8":
        value[[half - 1, 2 * half - 1]] = math.nan
    return torch.where(code >= half, -value, value)


def _values(codes, scales, form, cols):
    """What codes and scales stand for, in 32 bits."""
    rows, count = scales.shape
    if form == "fp4":
        codes = torch.stack((codes & 15, codes >> 4), dim=2)
    v = _table(form, codes.device)[codes.reshape(rows, count, BLOCK).int()]
    # 2^-127 is two factors: it is a denormal number
    e = scales.int().sub_(127).unsqueeze(2)
    v = torch.ldexp(torch.ldexp(v, e.div(2, rounding_mode="floor")),
                    e - e.div(2, rounding_mode="floor"))
    v = torch.where((scales == 255).unsqueeze(2), torch.full_like(v, math.nan), v)
    return v.reshape(rows, count * BLOCK)[:, :cols]


@functools.lru_cache(maxsize=None)
def _library(device):
    import sharded_mixed_precision_shard_amd as zs
    if zs.zs_init(device) != zs.ZS_OK:
        raise RuntimeError("zs_init")
    return zs


def run(s):
    op = s["op"]
    if own:
        zs = _library(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
        if op in ("save", "payload"):
            held = zs.Mx(s["codes"], s["scales"], s["cols"], s["form"])
            zs.zs_mx_quantize(s["in"], held, stream)
            if op == "payload":
                zs.zs_mx_dequantize(held, s["out"], stream)
        elif op == "linear":
            w = zs.Mx(s["codes"], s["scales"], s["k"], s["w"])
            zs.zs_mx_linear(s["in"], w, s["out"], stream, s["workspace"])
        elif op == "product":
            x = zs.Mx(s["xcodes"], s["xscales"], s["k"], s["x"])
            w = zs.Mx(s["codes"], s["scales"], s["k"], s["w"])
            zs.zs_mx_product(x, w, s["out"], stream, s["workspace"])
        elif op == "dgrad":
            w = zs.Mx(s["codes"], s["scales"], s["k"], s["w"])
            zs.zs_mx_linear_dgrad(s["in"], w, s["out"], stream, s["workspace"])
        else:
            x = zs.Mx(s["codes"], s["scales"], s["k"], s["x"])
            zs.zs_mx_linear_wgrad(s["in"], x, s["out"], s["add"], stream, s["workspace"])
    elif op in ("save", "payload"):
        codes, scales = _quantise(s["in"], s["form"])
        s["codes"].copy_(codes)
        s["scales"].copy_(scales)
        if op == "payload":
            s["out"].copy_(_values(codes, scales, s["form"], s["cols"]))
    elif op == "linear":
        w = _values(s["codes"], s["scales"], s["w"], s["k"])
        s["out"].copy_(s["in"].float() @ w.t())
    elif op == "product":
        x = _values(s["xcodes"], s["xscales"], s["x"], s["k"])
        w = _values(s["codes"], s["scales"], s["w"], s["k"])
        s["out"].copy_(x @ w.t())
    elif op == "dgrad":
        w = _values(s["codes"], s["scales"], s["w"], s["k"])
        s["out"].copy_(s["in"].float() @ w)
    else:
        x = _values(s["codes"], s["scales"], s["x"], s["k"])
        dw = s["in"].float().t() @ x
        s["out"].copy_(s["out"] + dw if s["add"] else dw)
    if op == "save":
        return {"values": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if op == "payload":
        return {"values": s["out"], "scales": s["scales"]}
    return s["out"]


def _exact_values(codes, scales, form, cols):
    """Decoded in 64 bits, code by code of the format's table."""
    if form == "fp4":
        sizes = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
        codes = torch.stack((codes % 16, codes // 16), 2).flatten(1)
    else:
        sizes = [i / 512.0 for i in range(8)]
        sizes += [(1 + i / 8.0) * 2.0 ** e for e in range(-6, 9) for i in range(8)]
        sizes[127] = math.nan
    table = torch.tensor(sizes + [-x for x in sizes], dtype=torch.float64, device=codes.device)
    factor = torch.tensor([2.0 ** (b - 127) for b in range(255)] + [math.nan],
                          dtype=torch.float64, device=codes.device)
    each = factor[scales.long()].repeat_interleave(BLOCK, 1)
    return (table[codes.long()] * each)[:, :cols]


def _exact_rounded(x, form):
    """(codes' values, the scales' powers) of the nearest codes of a [blocks, 32] matrix."""
    top = FORMS[form][0]
    x = x.double()
    peak = x.abs().max(1, keepdim=True).values
    factor = torch.exp2(torch.floor(torch.log2(peak)) - top)
    # log2 rounds: the peak's power is the largest that does not exceed it
    factor = torch.where(factor * 2.0 ** (top + 1) <= peak, factor * 2, factor)
    factor = torch.where(factor * 2.0 ** top > peak, factor / 2, factor).clamp(min=2.0 ** -127)
    if form == "fp4":
        sizes = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    else:
        sizes = [i / 512.0 for i in range(8)]
        sizes += [(1 + i / 8.0) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1]
    table = torch.tensor(sizes, dtype=torch.float64, device=x.device)
    between = (table[1:] + table[:-1]) / 2
    size = x.abs() / factor
    place = torch.searchsorted(between, size.contiguous())
    tie = between[place.clamp(max=len(sizes) - 2)] == size
    place = torch.where(tie & (place % 2 == 1), place + 1, place)
    return table[place.clamp(max=len(sizes) - 1)] * torch.sign(x), factor


def exact(case, seed):
    """The outputs of one pass in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("save", "payload"):
        rows, cols, form = case["rows"], case["cols"], case["form"]
        count = -(-cols // BLOCK)
        width = count * BLOCK if op == "save" else cols
        out = torch.zeros((rows, width), dtype=torch.float64, device=s["in"].device)
        high, wide = max(1, (1 << 25) // cols), min(cols, 1 << 25)
        for a in range(0, rows, high):
            for b in range(0, cols, wide):
                part = s["in"][a:a + high, b:b + wide].double()
                n = part.shape[1]
                full = torch.zeros((part.shape[0], -(-n // BLOCK) * BLOCK), dtype=torch.float64,
                                   device=part.device)
                full[:, :n] = part
                codes, factor = _exact_rounded(full.view(-1, BLOCK), form)
                if op == "payload":
                    codes = codes * factor
                codes = codes.view(full.shape)
                out[a:a + high, b:b + (n if op == "payload" else codes.shape[1])] = \
                    codes[:, :n] if op == "payload" else codes
        return {"values": out, "scales": None}
    form = case["x"] if op == "wgrad" else case["w"]
    held = _exact_values(s["codes"], s["scales"], form, case["k"])
    if op == "product":
        x = _exact_values(s["xcodes"], s["xscales"], case["x"], case["k"])
        return torch.mm(x, held.t())
    x = s["in"].double()
    if op == "linear":
        return torch.mm(x, held.t())
    if op == "dgrad":
        return torch.mm(x, held)
    grad = torch.mm(x.t(), held)
    return s["out"].double() + grad if case["add"] else grad


def work(case):
    """Bytes read once and written once, and floating-point operations."""

    def held(form, rows, cols):
        return rows * (_width(form, cols) + -(-cols // BLOCK))

    op = case["op"]
    if op in ("save", "payload"):
        rows, cols = case["rows"], case["cols"]
        size = torch.finfo(TYPES[case["type"]]).bits // 8 * rows * cols
        blocks = held(case["form"], rows, cols)
        if op == "save":
            return {"bytes": size + blocks, "flops": 3 * rows * cols}
        return {"bytes": 2 * size + 2 * blocks, "flops": 4 * rows * cols}
    m, n, k = case["m"], case["n"], case["k"]
    if op == "linear":
        size = 2 * m * k + held(case["w"], n, k) + 2 * m * n
    elif op == "product":
        size = held(case["x"], m, k) + held(case["w"], n, k) + 2 * m * n
    elif op == "dgrad":
        size = 2 * m * n + held(case["w"], n, k) + 2 * m * k
    else:
        size = 2 * m * n + held(case["x"], m, k)
        size += n * k * (2 if case["type"] == "bf16" else 8 if case["add"] else 4)
    return {"bytes": size, "flops": 2 * m * n * k}
