"""The products of a linear layer on microscaled operands where few calls go: NaN bytes and
codes through every kernel, powers of two at both ends, scales far apart, sums of many
splits, outputs of few rows or columns.  Inputs and tolerances as in test_gpu_mx_product.py:
whole numbers times powers of two give equal results, normals stay within C 2^-23 sum|p|."""
import ctypes

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _mx_reference as ref
from tests.test_gpu_mx_product import OPS, Case, held, plain
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def workspace(gpu):
    return zs.mx_workspace()


def sized(op, rows, other, depth):
    """(m, n, k) of a product whose output is [rows, other]."""
    return {"dgrad": (rows, depth, other), "wgrad": (depth, rows, other)}.get(
        op, (rows, other, depth))


def check_nan(torch, case, workspace, rows, cols):
    """NaN in these rows and columns of the output, and what was there before in the rest."""
    touched = np.zeros(case.shape, bool)
    touched[list(rows)] = True
    touched[:, list(cols)] = True
    for kind in (torch.bfloat16, torch.float32):
        for space in (None, workspace):
            _, out = case.out(kind)
            case.call(out, space)
            got = out.float().cpu().numpy()
            want = ref.bf16_round(case.want) if kind == torch.bfloat16 else \
                case.want.astype(np.float32)
            assert np.isnan(got[touched]).all()
            assert np.array_equal(got[~touched], want[~touched])


# few rows; tiles of 64 in four wave groups, of 32 and 64 by 128, of 128 in two and one, of 256
@pytest.mark.parametrize("size", [(8, 100, 600), (1, 40, 33), (90, 70, 300), (24, 130, 1200),
                                  (50, 24600, 264), (1100, 1530, 520), (2100, 2300, 256),
                                  (4100, 4360, 300)])
def test_nan_blocks_of_fp4_products(gpu, workspace, size):
    torch = gpu
    for seed in range(2):
        case = Case(torch, "product", *size, "fp4", True, seed, "fp4")
        blocks = case.a.scales.shape[1]
        i, j = size[0] // 2, size[1] // 3
        if seed == 0:
            case.a.scales[i, blocks // 2] = 255
            check_nan(torch, case, workspace, [i], [])
        else:
            case.b.scales[j, blocks - 1] = 255
            check_nan(torch, case, workspace, [], [j])


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("pad", [0, 1])
@pytest.mark.parametrize("size", [(3, 100, 600), (96, 70, 304), (304, 264, 600), (1100, 1536, 264)])
def test_nan_codes_of_fp8(gpu, workspace, op, pad, size):
    """E4M3's NaN, of either sign, in one element."""
    torch = gpu
    for code in (0x7F, 0xFF):
        case = Case(torch, op, *sized(op, *size), "fp8", True, 3, "fp8", pad)
        j, c = size[1] // 3, size[2] - 2
        if op in ("linear", "product"):
            case.b.codes[j, c] = code
        else:
            case.b.codes[c, j] = code
        check_nan(torch, case, workspace, [], [j])
    if op == "product":
        case = Case(torch, op, *size, "fp4", True, 3, "fp8")
        case.a.codes[size[0] // 2, 5] = 0x7F
        check_nan(torch, case, workspace, [size[0] // 2], [])


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("byte", [0, 1, 2, 20, 230, 250])
def test_bytes_at_both_ends(gpu, workspace, op, fmt, byte):
    """Every block's power of two near an end of its range, the other operand's numbers near
    the other: sums of whole numbers times 2^-1, exact."""
    torch = gpu
    power = byte - 127
    for n, (size, pad) in enumerate((((3, 72, 300), 0), ((40, 72, 304), 0), ((96, 104, 304), 1),
                                     ((304, 264, 520), 0))):
        case = Case(torch, op, *sized(op, *size), fmt, True, byte + n, ("fp4", "fp8")[n % 2], pad)
        old = case.b.scales.cpu().numpy()
        case.b.scales.fill_(byte)
        # the values again, without their blocks' own powers of two
        bv = ref.decode(case.b.codes.cpu().numpy(), np.full_like(old, 127), fmt, case.b.cols)
        if op == "product":
            other = min(254 - byte, 250)
            case.a.scales.fill_(other)
            av = ref.decode(case.a.codes.cpu().numpy(),
                            np.full(tuple(case.a.scales.shape), 127, np.uint8), case.a.format,
                            case.a.cols)
            shift = power + other - 127
        else:
            av = case.a.double().cpu().numpy()
            shift = -100 if power > 0 else 100
            case.a.mul_(2.0 ** shift)
            shift += power
        av, bv = (av.T if op == "wgrad" else av), (bv if op in ("dgrad", "wgrad") else bv.T)
        case.want = (av @ bv) * 2.0 ** shift
        for kind in (torch.float32, torch.bfloat16):
            for space in (None, workspace):
                _, out = case.out(kind)
                case.call(out, space)
                case.check_equal(out)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("rows", [3, 40, 300])
def test_fp8_elements_below_bf16(gpu, workspace, op, rows):
    """Elements of fewer than bf16's smallest denormal, 2^-133, are rounded to it in a product:
    each is off by at most half of that."""
    torch = gpu
    rng = np.random.default_rng(rows)
    size = sized(op, rows, 72, 304)
    case = Case(torch, op, *size, "fp8", True, rows, "fp8")
    codes = rng.integers(0, 64, tuple(case.b.codes.shape)).astype(np.uint8)
    codes[:, case.b.cols:] = 0
    scales = rng.integers(0, 4, tuple(case.b.scales.shape)).astype(np.uint8)
    case.b.codes.copy_(torch.from_numpy(codes))
    case.b.scales.copy_(torch.from_numpy(scales))
    if op == "product":
        case.a.scales.fill_(240)
        av = ref.decode(case.a.codes.cpu().numpy(), case.a.scales.cpu().numpy(), "fp8", case.a.cols)
    else:
        case.a.mul_(2.0 ** 110)
        av = case.a.double().cpu().numpy()
    bv = ref.decode(codes, scales, "fp8", case.b.cols)
    av, bv = (av.T if op == "wgrad" else av), (bv if op in ("dgrad", "wgrad") else bv.T)
    want, sizes = av @ bv, np.abs(av) @ np.abs(bv)
    lost = np.abs(av).sum(1, keepdims=True) * 2.0 ** -134
    for space in (None, workspace):
        _, out = case.out(torch.float32)
        case.call(out, space)
        room = case.depth * 2.0 ** -23 * (sizes + lost) + lost
        assert (np.abs(out.double().cpu().numpy() - want) <= room).all()


@pytest.mark.parametrize("spread", [10, 60])
@pytest.mark.parametrize("rows", [1, 8, 16])
def test_few_rows_of_scales_far_apart(gpu, workspace, spread, rows):
    """Powers of two that differ by up to 2^120 in one sum.  In any order a partial sum is at
    most the sum of the magnitudes, so sums are within the bound where that is below 2^127;
    the others may pass the end of fp32."""
    torch = gpu
    rng = np.random.default_rng(rows)
    for xfmt, wfmt in (("fp4", "fp4"), ("fp8", "fp4"), ("fp4", "fp8")):
        case = Case(torch, "product", rows, 100, 1300, wfmt, False, rows, xfmt)
        for mx in (case.a, case.b):
            s = rng.integers(127 - spread, 128 + spread, tuple(mx.scales.shape)).astype(np.uint8)
            mx.scales.copy_(torch.from_numpy(s))
        a, b = (ref.decode(x.codes.cpu().numpy(), x.scales.cpu().numpy(), x.format, x.cols)
                for x in (case.a, case.b))
        want, sizes = a @ b.T, np.abs(a) @ np.abs(b.T)
        fits = sizes < 2.0 ** 127
        assert fits.mean() > 0.8
        case.want, case.sizes = want[fits], sizes[fits]
        for kind in (torch.float32, torch.bfloat16):
            for space in (None, workspace):
                _, out = case.out(kind)
                case.call(out, space)
                case.check_near(out[torch.from_numpy(fits).cuda()])


@pytest.mark.parametrize("op,size", [
    ("linear", (1, 200, 65536)), ("linear", (72, 200, 16384)), ("linear", (70, 200, 16389)),
    ("product", (1, 200, 65536)), ("product", (72, 200, 32768)),
    ("dgrad", (72, 16384, 200)), ("dgrad", (70, 16391, 201)),
    ("wgrad", (16384, 72, 200)), ("wgrad", (16391, 70, 201))])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_many_splits_give_the_same_bits(gpu, op, size, fmt):
    """Five splits and more, whose sums round: the order in which they end does not show, with
    other work beside them or without."""
    torch = gpu
    case = Case(torch, op, *size, fmt, False, 1)
    space, side = zs.mx_workspace(), torch.cuda.Stream()
    _, first = case.out(torch.float32)
    case.call(first, space)
    case.check_near(first)
    assert space[65536:].any()                     # sums went through the workspace
    busy = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for n in range(8):
        if n % 2:
            with torch.cuda.stream(side):
                busy = busy.mul(1.0001)
        _, out = case.out(torch.float32)
        case.call(out, space)
        assert torch.equal(out, first)
    torch.cuda.synchronize()
    assert not space[:65536].any()


@pytest.mark.parametrize("op,size", [
    ("linear", (64, 262200, 256)), ("linear", (130, 131100, 257)), ("product", (100, 168000, 257)),
    ("dgrad", (262149, 40, 64)), ("dgrad", (70, 40, 262200)), ("wgrad", (40, 64, 262200)),
    ("wgrad", (40, 262200, 64))])
def test_outputs_of_few_rows_or_columns(gpu, workspace, op, size):
    """As many elements as the largest tiles are for, but fewer rows or columns than a tile."""
    torch = gpu
    case = Case(torch, op, *size, "fp8" if op == "wgrad" else "fp4", True, 6)
    flat, out = case.out(torch.bfloat16, 8)
    before = flat.clone()
    case.call(out, workspace)
    case.check_equal(out)
    out.fill_(55.0)
    assert torch.equal(flat, before)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["bfloat16", "float16", "float32"])
def test_streamed_casts_equal_small_ones(gpu, fmt, kind):
    """Matrices that the casts stream, against the same rows a few at a time."""
    torch = gpu
    dtype = getattr(torch, kind)
    for rows, cols in ((17, 1000003), (14, 10_000_000)):
        gen = torch.Generator(device="cuda").manual_seed(rows)
        x = torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(generator=gen)
        x[rows // 2, cols // 3] = float("nan")
        whole = zs.Mx.empty(rows, cols, fmt)
        back = torch.empty_like(x)
        s = torch.cuda.current_stream()
        zs.zs_mx_quantize(x, whole, s)
        zs.zs_mx_dequantize(whole, back, s)
        step = 1 << 20                                   # elements of a part, whole blocks
        for row in (0, rows // 2, rows - 1):
            for a in range(0, cols, step):
                b = min(a + step, cols)
                part = zs.Mx.empty(1, b - a, fmt)
                value = torch.empty(b - a, dtype=dtype, device="cuda")
                zs.zs_mx_quantize(x[row, a:b], part, s)
                zs.zs_mx_dequantize(part, value, s)
                each = zs.mx_row_bytes(fmt, 32)
                first, last = a // 32, -(-b // 32)
                assert torch.equal(whole.codes[row, first * each:last * each], part.codes[0])
                assert torch.equal(whole.scales[row, first:last], part.scales[0])
                assert torch.equal(back[row, a:b].view(torch.uint8), value.view(torch.uint8))


@pytest.mark.parametrize("xfmt,wfmt,rows,n", [
    ("fp4", "fp4", 1, 2 ** 27 + 5), ("fp8", "fp4", 17, 2 ** 27 + 21), ("fp4", "fp8", 2, 2 ** 28),
    ("fp4", "fp4", 33, 2 ** 27), ("fp4", "fp4", 3, 2 ** 27 - 16)])
def test_more_columns_than_a_grid_dimension_holds(gpu, xfmt, wfmt, rows, n):
    """A few rows through as many rows of w as the library takes: strips of 16 of them with
    512 threads each are 2^32 threads from 2^27 on.  Zeros but for rows near both ends and at
    the border."""
    torch = gpu
    rng = np.random.default_rng(rows)
    x, xv = held(torch, rng, rows, 32, xfmt, True)
    at = {0, 15, 16, 2 ** 26 + 1, 2 ** 27 - 17, 2 ** 27 - 16, 2 ** 27 - 1, n - 2, n - 1}
    at = sorted(i for i in at if i < n)
    few, wv = held(torch, rng, len(at), 32, wfmt, True)
    w = zs.Mx.empty(n, 32, wfmt)
    w.codes.zero_()
    w.scales.fill_(127)
    where = torch.tensor(at, device="cuda")
    w.codes[where] = few.codes
    w.scales[where] = few.scales
    y = torch.full((rows, n), 7.0, dtype=torch.bfloat16, device="cuda")
    zs.zs_mx_product(x, w, y, torch.cuda.current_stream())
    want = ref.bf16_round(xv @ wv.T)
    assert np.array_equal(y[:, where].float().cpu().numpy(), want)
    y[:, where] = 0.0
    assert not y.any()


@pytest.mark.parametrize("rows", [2 ** 32 - 1, 2 ** 32 - 256])
def test_casts_of_as_many_blocks_as_one_call_takes(gpu, rows):
    """A column of 2^32 - 1 elements is as many blocks.  Zeros but for its ends and the borders
    of a grid's dimension."""
    torch = gpu
    rng = np.random.default_rng(1)
    at = [0, 255, 256, 2 ** 31 - 1, 2 ** 31, 2 ** 32 - 258, rows - 257, rows - 256, rows - 2,
          rows - 1]
    at = sorted(set(at))
    values = rng.choice([-3.0, -1.0, 0.5, 1.5, 6.0], len(at))
    x = torch.zeros(rows, 1, dtype=torch.bfloat16, device="cuda")
    for i, v in zip(at, values):
        x[i] = v
    q = zs.Mx.empty(rows, 1, "fp4")
    zs.zs_mx_quantize(x, q, torch.cuda.current_stream())
    codes, scales = ref.encode(values[:, None], "fp4")
    for n, i in enumerate(at):
        assert np.array_equal(q.codes[i].cpu().numpy(), codes[n])
        assert q.scales[i].item() == scales[n, 0]
    x.fill_(7.0)
    zs.zs_mx_dequantize(q, x, torch.cuda.current_stream())
    for i, v in zip(at, values):
        assert x[i].item() == v
        x[i] = 0.0
    part = 2 ** 28
    assert not any(x[i:i + part].any().item() for i in range(0, rows, part))


@pytest.mark.parametrize("ld", [2 ** 22, 2 ** 54, 2 ** 55, 3 * 2 ** 54, 2 ** 58])
def test_one_row_of_any_distance(gpu, workspace, ld):
    """A single row has no next one, and its distance to that may be any number."""
    torch = gpu
    for op, size in (("dgrad", (1, 264, 320)), ("wgrad", (1, 264, 320)), ("linear", (1, 264, 320))):
        case = Case(torch, op, *size, "fp4", True, 2)
        _, out = case.out(torch.float32)
        a = zs.ZsMatrix(case.a.data_ptr(), 1, case.a.shape[1], ld, 0, 0)
        to = zs._matrix(out, "out")
        lib, stream = zs.load_library(), torch.cuda.current_stream().cuda_stream
        args = [ctypes.byref(a), case.b.ref, ctypes.byref(to)]
        if op == "wgrad":
            args.append(0)
        call = lib.zs_mx_linear if op == "linear" else getattr(lib, "zs_mx_linear_" + op)
        assert call(*args, workspace.data_ptr(), stream) == zs.ZS_OK
        case.check_equal(out)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("rows", [3, 40, 300])
@pytest.mark.parametrize("byte", [246, 250, 252, 253, 254])
def test_bytes_past_those_of_finite_inputs(gpu, workspace, op, fmt, rows, byte):
    """Bytes that no finite bf16 matrix is quantised to: elements past bf16's largest are
    infinite in a product, but for fp4 x fp4, which takes the codes themselves.  One element of
    the depth is not zero, and each column of the output has another code there."""
    torch = gpu
    case = Case(torch, op, *sized(op, rows, 264, 304), fmt, True, 2, "fp4")
    case.b.codes.zero_()
    case.b.scales.fill_(byte)
    codes = np.arange(264) % (16 if fmt == "fp4" else 256)
    codes[np.isnan(ref.code_values(fmt)[codes])] = 0
    column = torch.from_numpy(codes.astype(np.uint8)).cuda()
    if op in ("linear", "product"):
        case.b.codes[:, 0] = column
    elif fmt == "fp4":
        case.b.codes[0, :132] = column[0::2] | (column[1::2] << 4)
    else:
        case.b.codes[0, :264] = column
    if op == "product":
        case.a.codes.fill_(0x22)                        # ones, times 2^-40
        case.a.codes[:, 304 // 2:] = 0
        case.a.scales.fill_(127 - 40)
    else:
        case.a.fill_(2.0 ** -40)
    values = ref.code_values(fmt)[codes] * 2.0 ** (byte - 127)
    if not (op == "product" and fmt == "fp4"):
        past = np.abs(values) > 2.0 ** 128 - 2.0 ** 120          # bf16's largest
        values = np.where(past, np.copysign(np.inf, values), values)
    case.want = np.broadcast_to(values * 2.0 ** -40, case.shape)
    for space in (None, workspace):
        _, out = case.out(torch.float32)
        case.call(out, space)
        assert np.array_equal(out.cpu().numpy(), case.want.astype(np.float32))
