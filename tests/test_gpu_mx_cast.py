"""Quantisation into the microscaled formats and back on the GPU, against a plain
implementation in 64 bits.  Codes and scales are whole numbers that the
definition fixes: equal.  Values read back are the code times a power of two,
rounded once: equal to that rounding, NaN where the block is NaN."""
import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _mx_reference as ref
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

TYPES = ("bfloat16", "float16", "float32")
SIZES = [(1, 1), (1, 31), (1, 32), (3, 33), (7, 8), (2, 4096), (37, 1001), (129, 96), (1, 100003),
         (1025, 40), (300, 512)]


def inputs(torch, rows, cols, kind, seed, wild=False):
    """A matrix of normals, rows of different magnitudes, in the type's range."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols))
    span = 8 if kind == "float16" else 60
    x *= np.exp2(rng.integers(-span, span, (rows, 1)).astype(float))
    x[rng.random((rows, cols)) < 0.05] = 0.0
    if wild:
        x[rng.random((rows, cols)) < 0.01] = np.inf
        x[rng.random((rows, cols)) < 0.01] = np.nan
        x[rng.random((rows, cols)) < 0.01] = -np.inf
    with np.errstate(all="ignore"):
        return torch.from_numpy(x.astype(np.float32)).to(getattr(torch, kind))


def strided(torch, x, pad, offset):
    """x on the GPU with rows pad elements further apart, offset elements into memory."""
    rows, cols = x.shape
    flat = torch.full((offset + rows * (cols + pad) + 64,), 77.0, dtype=x.dtype, device="cuda")
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return flat, view


def check_codes(torch, held, x, fmt):
    codes, scales = ref.encode(x.double().numpy(), fmt)
    assert np.array_equal(held.scales.cpu().numpy(), scales)
    got = held.codes.cpu().numpy()
    assert np.array_equal(got, codes)
    return codes, scales


def check_values(torch, got, codes, scales, fmt, cols, kind):
    want = torch.from_numpy(ref.decode(codes, scales, fmt, cols))
    if kind == "bfloat16":   # via binary32, exact for a code times a power of two
        want = want.float().to(torch.bfloat16)
    else:
        want = want.to(getattr(torch, kind))
    got = got.cpu()
    nan = torch.isnan(want.float())
    assert torch.equal(torch.isnan(got.float()), nan)
    assert torch.equal(torch.where(nan, torch.zeros_like(got), got),
                       torch.where(nan, torch.zeros_like(want), want))


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1), (8, 8)])
def test_round_trip(gpu, fmt, kind, pad, offset):
    torch = gpu
    for n, (rows, cols) in enumerate(SIZES):
        x = inputs(torch, rows, cols, kind, n, wild=n % 2 == 1)
        _, view = strided(torch, x, pad, offset)
        held = zs.Mx.empty(rows, cols, fmt)
        zs.zs_mx_quantize(view, held, torch.cuda.current_stream())
        codes, scales = check_codes(torch, held, x, fmt)
        for to in TYPES:
            flat, out = strided(torch, torch.zeros(rows, cols, dtype=getattr(torch, to)), pad,
                                offset)
            before = flat.clone()
            zs.zs_mx_dequantize(held, out, torch.cuda.current_stream())
            check_values(torch, out, codes, scales, fmt, cols, to)
            # the gaps between rows and what lies around are left as they were
            out.zero_()
            assert torch.equal(flat, before)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_bf16(gpu, fmt):
    """Every bf16 value, in blocks with a companion that fixes the scale, and alone."""
    torch = gpu
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    values = bits.view(torch.bfloat16)
    x = torch.zeros(65536, 32, dtype=torch.bfloat16)
    x[:, 5] = values
    for companion in (None, 1.0, 6.5, 2.0 ** 100, 2.0 ** -126):
        if companion is not None:
            x[:, 6] = companion
        held = zs.Mx.empty(65536, 32, fmt)
        zs.zs_mx_quantize(x.cuda(), held, torch.cuda.current_stream())
        codes, scales = check_codes(torch, held, x, fmt)
        for to in TYPES:
            out = torch.empty(65536, 32, dtype=getattr(torch, to), device="cuda")
            zs.zs_mx_dequantize(held, out, torch.cuda.current_stream())
            check_values(torch, out, codes, scales, fmt, 32, to)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_ties_and_neighbours(gpu, fmt):
    """Every midpoint of two codes, and the binary32 numbers beside it, at three scales."""
    torch = gpu
    table = ref.SIZES[fmt]
    mid = (table[1:] + table[:-1]) / 2
    past = [6.5, 7.0, 7.5] if fmt == "fp4" else [460.0, 464.0, 511.0]
    points = np.concatenate((table, mid, past))
    points = points.astype(np.float32)
    points = np.concatenate((points, np.nextafter(points, np.float32(1e9)),
                             np.nextafter(points, np.float32(-1))))
    x = np.zeros((len(points) * 2, 32), np.float32)
    x[:, 0] = np.concatenate((points, -points))
    x[:, 31] = table[-1]
    x = np.concatenate([x * np.float32(2.0 ** e) for e in (0, 90, -100)])
    x = torch.from_numpy(x)
    held = zs.Mx.empty(x.shape[0], 32, fmt)
    zs.zs_mx_quantize(x.cuda(), held, torch.cuda.current_stream())
    check_codes(torch, held, x, fmt)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_code_and_scale_reads_back(gpu, fmt):
    torch = gpu
    half = np.arange(256, dtype=np.uint8)
    codes = np.tile(half.reshape(-1, ref.row_bytes(fmt, 32)), (256, 1))
    scales = np.repeat(half, codes.shape[0] // 256).reshape(-1, 1)
    held = zs.Mx(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32, fmt)
    for to in TYPES:
        out = torch.empty(held.rows, 32, dtype=getattr(torch, to), device="cuda")
        zs.zs_mx_dequantize(held, out, torch.cuda.current_stream())
        check_values(torch, out, codes, scales, fmt, 32, to)


def test_flat_shard_and_its_parts(gpu):
    """A long row holds the blocks of the matrices inside it."""
    torch = gpu
    flat = inputs(torch, 1, 64 * 96 + 32 + 33 * 64 + 7, "bfloat16", 5)[0].cuda()
    held = zs.Mx.empty(1, flat.numel(), "fp4")
    zs.zs_mx_quantize(flat, held, torch.cuda.current_stream())
    for start, rows, cols in ((0, 64, 96), (64 * 96 + 32, 33, 64), (32, 1, 32), (64, 0, 32)):
        part = held.part(start, rows, cols)
        own = zs.Mx.empty(rows, cols, "fp4")
        zs.zs_mx_quantize(flat[start:start + rows * cols].view(rows, cols), own,
                          torch.cuda.current_stream())
        assert torch.equal(part.codes, own.codes) and torch.equal(part.scales, own.scales)
    # 16-bit integers are bf16 patterns, as the step's parameter copy may be held
    again = zs.Mx.empty(1, flat.numel(), "fp4")
    zs.zs_mx_quantize(flat.view(torch.int16), again, torch.cuda.current_stream())
    assert torch.equal(again.codes, held.codes)
    for bad in ((1, 1, 32), (0, 1, 33), (0, 1000, 32), (-32, 1, 32)):
        with pytest.raises(ValueError):
            held.part(*bad)


def test_nothing_to_do(gpu):
    torch = gpu
    for rows, cols in ((0, 32), (5, 0), (0, 0)):
        held = zs.Mx.empty(rows, cols, "fp8")
        x = torch.empty(rows, cols, device="cuda")
        assert zs.zs_mx_quantize(x, held) == zs.ZS_OK
        assert zs.zs_mx_dequantize(held, x) == zs.ZS_OK


def test_more_than_2_32_elements(gpu):
    """Offsets past 32 bits: a row of 2^32 + 96 elements, checked at its ends."""
    torch = gpu
    n = 2 ** 32 + 96
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    edge = inputs(torch, 1, 4096, "bfloat16", 9)[0]
    x[:4096] = edge.cuda()
    x[n - 4096:] = edge.cuda()
    held = zs.Mx.empty(1, n, "fp4")
    zs.zs_mx_quantize(x, held, torch.cuda.current_stream())
    codes, scales = ref.encode(edge.double().numpy()[None], "fp4")
    for part in (held.part(0, 1, 4096), held.part(n - 4096, 1, 4096)):
        assert np.array_equal(part.codes.cpu().numpy(), codes)
        assert np.array_equal(part.scales.cpu().numpy(), scales)
    x.zero_()
    zs.zs_mx_dequantize(held, x, torch.cuda.current_stream())
    want = torch.from_numpy(ref.decode(codes, scales, "fp4", 4096)[0]).to(torch.bfloat16)
    assert torch.equal(x[:4096].cpu(), want) and torch.equal(x[n - 4096:].cpu(), want)
