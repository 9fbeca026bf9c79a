"""The linear layer on microscaled operands at the ends of its sizes, and on operands that lie
where only some callers put them.  Sums of whole numbers: results are equal to the exact ones."""
import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _mx_reference as ref
from tests.test_gpu_mx_product import OPS, Case, held, plain
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

TOP = 2 ** 28          # M, N and K up to this


@pytest.fixture(scope="module")
def workspace(gpu):
    gpu.cuda.empty_cache()
    yield zs.mx_workspace()
    gpu.cuda.empty_cache()


def blocks(torch, rows, cols, fmt):
    """An Mx of zeros."""
    x = zs.Mx.empty(rows, cols, fmt)
    x.codes.zero_()
    x.scales.fill_(127)
    return x


def put_columns(torch, to, first, part):
    """The blocks of ``part`` from column ``first`` on, a multiple of 32."""
    each = zs.mx_row_bytes(to.format, 32)
    a, n = first // 32, part.scales.shape[1]
    to.codes[:, a * each:(a + n) * each] = part.codes
    to.scales[:, a:a + n] = part.scales


@pytest.mark.parametrize("op,rows,xfmt,fmt", [
    ("linear", 1, "", "fp4"), ("linear", 17, "", "fp4"), ("linear", 1, "", "fp8"),
    ("product", 1, "fp4", "fp4"), ("product", 17, "fp4", "fp4"), ("product", 2, "fp8", "fp4"),
    ("product", 65, "fp8", "fp4")])
@pytest.mark.parametrize("depth", [2 ** 24 + 96, TOP])
def test_rows_as_long_as_they_may_be(gpu, workspace, op, rows, xfmt, fmt, depth):
    """Zeros but for 96 columns at both ends."""
    torch = gpu
    if rows == 65 and depth == TOP:
        rows = 20                                  # 65 such rows of bytes are 17 GB
    rng = np.random.default_rng(rows)
    w, want, n = blocks(torch, 3, depth, fmt), 0.0, 96
    if op == "linear":
        x = torch.zeros(rows, depth, dtype=torch.bfloat16, device="cuda")
    else:
        x = blocks(torch, rows, depth, xfmt)
    for at in (0, depth - n):
        wp, wv = held(torch, rng, 3, n, fmt, True)
        put_columns(torch, w, at, wp)
        if op == "linear":
            xp, xv = plain(torch, rng, rows, n, True, 0, 0)
            x[:, at:at + n] = xp
        else:
            xp, xv = held(torch, rng, rows, n, xfmt, True)
            put_columns(torch, x, at, xp)
        want = want + xv @ wv.T
    y = torch.full((rows, 3), 7.0, device="cuda")
    call = zs.zs_mx_linear if op == "linear" else zs.zs_mx_product
    call(x, w, y, torch.cuda.current_stream(), workspace)
    assert np.array_equal(y.cpu().numpy(), want.astype(np.float32))
    assert not workspace[:65536].any()


@pytest.mark.parametrize("op", ["dgrad", "wgrad"])
@pytest.mark.parametrize("rows", [1, 8, 3])
def test_sums_over_as_many_rows_as_there_may_be(gpu, workspace, op, rows):
    """Depth 2^28, zeros but for 64 rows at both ends."""
    torch = gpu
    rng = np.random.default_rng(rows)
    fmt = "fp4" if op == "dgrad" else "fp8"
    q, want = blocks(torch, TOP, 32, fmt), 0.0
    p = torch.zeros((rows, TOP) if op == "dgrad" else (TOP, rows), dtype=torch.bfloat16,
                    device="cuda")
    for at in (0, TOP - 64):
        qp, qv = held(torch, rng, 64, 32, fmt, True)
        q.codes[at:at + 64], q.scales[at:at + 64] = qp.codes, qp.scales
        if op == "dgrad":
            pp, pv = plain(torch, rng, rows, 64, True, 0, 0)
            p[:, at:at + 64] = pp
        else:
            pp, pv = plain(torch, rng, 64, rows, True, 0, 0)
            p[at:at + 64], pv = pp, pv.T
        want = want + pv @ qv
    out = torch.full((rows, 32), 7.0, device="cuda")
    if op == "dgrad":
        zs.zs_mx_linear_dgrad(p, q, out, torch.cuda.current_stream(), workspace)
    else:
        zs.zs_mx_linear_wgrad(p, q, out, False, torch.cuda.current_stream(), workspace)
    assert np.array_equal(out.cpu().numpy(), want.astype(np.float32))


@pytest.mark.parametrize("op", ["linear", "product", "dgrad", "wgrad"])
def test_outputs_of_as_many_rows_as_there_may_be(gpu, workspace, op):
    """2^28 rows of three columns, zeros but for six near the ends and the middle."""
    torch = gpu
    rng = np.random.default_rng(1)
    at = torch.tensor([0, 255, 2 ** 27 - 1, 2 ** 27, TOP - 257, TOP - 1], device="cuda")
    y = torch.full((TOP, 3), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.current_stream()
    if op in ("linear", "product"):
        w, wv = held(torch, rng, 3, 32, "fp4", True)
        if op == "linear":
            xp, xv = plain(torch, rng, 6, 32, True, 0, 0)
            x = torch.zeros(TOP, 32, dtype=torch.bfloat16, device="cuda")
            x[at] = xp
            zs.zs_mx_linear(x, w, y, s, workspace)
        else:
            xp, xv = held(torch, rng, 6, 32, "fp4", True)
            x = blocks(torch, TOP, 32, "fp4")
            x.codes[at], x.scales[at] = xp.codes, xp.scales
            zs.zs_mx_product(x, w, y, s, workspace)
        want = xv @ wv.T
    elif op == "dgrad":
        w, wv = held(torch, rng, 2, 3, "fp4", True)
        dp, dv = plain(torch, rng, 6, 2, True, 0, 0)
        dy = torch.zeros(TOP, 2, dtype=torch.bfloat16, device="cuda")
        dy[at] = dp
        zs.zs_mx_linear_dgrad(dy, w, y, s, workspace)
        want = dv @ wv
    else:
        x, xv = held(torch, rng, 2, 3, "fp8", True)
        dp, dv = plain(torch, rng, 2, 6, True, 0, 0)
        dy = torch.zeros(2, TOP, dtype=torch.bfloat16, device="cuda")
        dy[:, at] = dp
        zs.zs_mx_linear_wgrad(dy, x, y, False, s, workspace)
        want = dv.T @ xv
    assert np.array_equal(y[at].float().cpu().numpy(), ref.bf16_round(want))
    y[at] = 0.0
    assert not y.any()


@pytest.mark.parametrize("op", ["dgrad", "wgrad"])
def test_outputs_of_as_many_columns_as_there_may_be(gpu, workspace, op):
    torch = gpu
    rng = np.random.default_rng(2)
    q, want, s = blocks(torch, 2, TOP, "fp4"), [], torch.cuda.current_stream()
    p, pv = plain(torch, rng, *((3, 2) if op == "dgrad" else (2, 3)), True, 0, 0)
    for at in (0, 2 ** 27, TOP - 64):
        qp, qv = held(torch, rng, 2, 64, "fp4", True)
        put_columns(torch, q, at, qp)
        want.append((at, (pv if op == "dgrad" else pv.T) @ qv))
    out = torch.full((3, TOP), 7.0, dtype=torch.bfloat16, device="cuda")
    if op == "dgrad":
        zs.zs_mx_linear_dgrad(p, q, out, s, workspace)
    else:
        zs.zs_mx_linear_wgrad(p, q, out, False, s, workspace)
    for at, v in want:
        assert np.array_equal(out[:, at:at + 64].float().cpu().numpy(), ref.bf16_round(v))
        out[:, at:at + 64] = 0.0
    assert not out.any()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("skip", [1, 3, 6])
def test_blocks_inside_a_shard(gpu, workspace, op, fmt, skip):
    """A weight's blocks as they lie in a long row: its scales begin at any byte."""
    torch = gpu
    for size in ((3, 72, 544), (40, 72, 288), (130, 136, 544)):
        size = {"dgrad": (size[0], size[2], 96), "wgrad": (size[2], size[0], 96)}.get(op, size)
        case = Case(torch, op, *size, fmt, True, skip, fmt)
        own = case.b
        flat = blocks(torch, 1, 32 * skip + own.rows * own.cols + 64, fmt)
        case.b = flat.part(32 * skip, own.rows, own.cols)
        case.b.codes.copy_(own.codes)
        case.b.scales.copy_(own.scales)
        assert case.b.codes.data_ptr() != own.codes.data_ptr()
        for space in (None, workspace):
            _, out = case.out(torch.float32)
            case.call(out, space)
            case.check_equal(out)


@pytest.mark.parametrize("rows", [5, 40, 300])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_an_operand_with_itself(gpu, workspace, rows, fmt):
    torch = gpu
    x, xv = held(torch, np.random.default_rng(rows), rows, 520, fmt, True)
    y = torch.empty(rows, rows, device="cuda")
    zs.zs_mx_product(x, x, y, torch.cuda.current_stream(), workspace)
    assert np.array_equal(y.cpu().numpy(), (xv @ xv.T).astype(np.float32))


@pytest.mark.parametrize("op", ["linear", "dgrad", "wgrad"])
@pytest.mark.parametrize("rows,pad", [(3, 0), (40, 0), (40, 1), (304, 0)])
def test_denormal_activations(gpu, workspace, op, rows, pad):
    """bf16 denormals, whole multiples of 2^-133, against powers of two that make them normal."""
    torch = gpu
    size = {"dgrad": (rows, 304, 72), "wgrad": (304, rows, 72)}.get(op, (rows, 72, 304))
    case = Case(torch, op, *size, "fp4", True, rows, pad=pad)
    case.want = case.want * 2.0 ** (100 - 133)
    case.a.mul_(2.0 ** -66).mul_(2.0 ** -67)
    assert (case.a.float().abs().max() <= 8 * 2.0 ** -133).item() and case.a.any()
    case.b.scales.add_(100)
    for kind in (torch.float32, torch.bfloat16):
        _, out = case.out(kind)
        case.call(out, workspace)
        case.check_equal(out)
