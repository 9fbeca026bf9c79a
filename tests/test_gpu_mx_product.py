"""The linear layer on microscaled operands and its backward products on the GPU,
against products of the decoded operands in 64 bits.

Two kinds of inputs.  Whole numbers times small powers of two, where every sum
is exact in binary32 whatever its order: the fp32 output is equal to the exact
one, the bf16 output to its rounding.  And normals, where the tolerance is what
fp32 sums of C products can be off by: the products are exact (8 and at most 8
bits), each of at most C additions is off by at most 2^-23 of the magnitudes'
sum (a truncating adder; half of it where it rounds), so by C 2^-23 sum|p| in
all; a bf16 output adds half a step, 2^-8 of the value."""
import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _mx_reference as ref
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

OPS = ("linear", "product", "dgrad", "wgrad")
# rows of the activation, rows and columns of the weight
SIZES = [(1, 1, 1), (1, 16, 32), (2, 5, 40), (3, 33, 31), (5, 64, 65), (17, 48, 96),
         (37, 100, 129), (64, 64, 64), (65, 130, 200), (130, 257, 96), (200, 300, 513),
         (129, 127, 1000), (260, 520, 264)]


@pytest.fixture(scope="module")
def workspace(gpu):
    return zs.mx_workspace()


def held(torch, rng, rows, cols, fmt, exact):
    """An operand in blocks, on the GPU, and its values in 64 bits."""
    if exact:
        # multiples of 1/2 up to 6, or whole numbers up to 15, times 2^-1 .. 2
        top = ref.FP4 if fmt == "fp4" else np.arange(16.0)
        values = rng.choice(top, (rows, cols)) * rng.choice([-1.0, 1.0], (rows, cols))
        nb = -(-cols // 32)
        full = np.zeros((rows, nb * 32))
        full[:, :cols] = values
        table = ref.code_values(fmt)[:8 if fmt == "fp4" else 127]
        codes = np.searchsorted(table, np.abs(full)).astype(np.uint8)
        codes += np.where(full < 0, 8 if fmt == "fp4" else 128, 0).astype(np.uint8)
        if fmt == "fp4":
            codes = codes[:, 0::2] | (codes[:, 1::2] << 4)
        codes = np.ascontiguousarray(codes)
        scales = rng.integers(126, 129, (rows, nb)).astype(np.uint8)
    else:
        x = rng.standard_normal((rows, cols)) * np.exp2(rng.integers(-3, 4, (rows, 1)))
        codes, scales = ref.encode(x, fmt)
    mx = zs.Mx(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), cols, fmt)
    return mx, ref.decode(codes, scales, fmt, cols)


def plain(torch, rng, rows, cols, exact, pad, offset):
    """A bf16 operand with rows pad apart, NaN in the gaps, and its values."""
    x = rng.integers(-8, 9, (rows, cols)).astype(float) if exact else \
        rng.standard_normal((rows, cols))
    x = torch.from_numpy(x).to(torch.bfloat16)
    flat = torch.full((offset + rows * (cols + pad) + 64,), float("nan"), dtype=torch.bfloat16,
                      device="cuda")
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    return view, x.double().numpy()


class Case:
    """One product: its inputs, its call, and the exact result."""

    def __init__(self, torch, op, m, n, k, fmt, exact, seed, xfmt="fp4", pad=0, offset=0):
        rng = np.random.default_rng(seed)
        self.torch, self.op = torch, op
        if op == "linear":
            a, av = plain(torch, rng, m, k, exact, pad, offset)
            b, bv = held(torch, rng, n, k, fmt, exact)
            self.shape, bv = (m, n), bv.T
        elif op == "product":
            a, av = held(torch, rng, m, k, xfmt, exact)
            b, bv = held(torch, rng, n, k, fmt, exact)
            self.shape, bv = (m, n), bv.T
        elif op == "dgrad":
            a, av = plain(torch, rng, m, n, exact, pad, offset)
            b, bv = held(torch, rng, n, k, fmt, exact)
            self.shape = (m, k)
        else:
            a, av = plain(torch, rng, m, n, exact, pad, offset)
            b, bv = held(torch, rng, m, k, fmt, exact)
            self.shape, av = (n, k), av.T
        self.a, self.b, self.depth = a, b, bv.shape[0]
        # a long sum in pieces keeps every partial sum exact where the inputs are
        self.want = av @ bv
        self.sizes = np.abs(av) @ np.abs(bv)

    def out(self, kind, pad=0, offset=0, fill=None):
        """(all of the memory, the output inside it)."""
        torch = self.torch
        rows, cols = self.shape
        flat = torch.full((offset + rows * (cols + pad) + 64,), 55.0, dtype=kind, device="cuda")
        view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        if fill is not None:
            view.copy_(torch.from_numpy(fill))
        return flat, view

    def call(self, out, workspace=None, add=False, stream=None):
        s = stream or self.torch.cuda.current_stream()
        if self.op == "linear":
            zs.zs_mx_linear(self.a, self.b, out, s, workspace)
        elif self.op == "product":
            zs.zs_mx_product(self.a, self.b, out, s, workspace)
        elif self.op == "dgrad":
            zs.zs_mx_linear_dgrad(self.a, self.b, out, s, workspace)
        else:
            zs.zs_mx_linear_wgrad(self.a, self.b, out, add, s, workspace)

    def check_equal(self, out, more=0.0):
        got = out.float().cpu().numpy()
        want = self.want + more
        want = ref.bf16_round(want) if out.dtype == self.torch.bfloat16 else want.astype(np.float32)
        assert np.array_equal(got, want), (self.op, self.shape, np.argwhere(got != want)[:5])

    def check_near(self, out):
        got = out.double().cpu().numpy()
        room = self.depth * 2.0 ** -23 * self.sizes
        if out.dtype == self.torch.bfloat16:
            room = room + 2.0 ** -8 * (np.abs(self.want) + room)
        off = np.abs(got - self.want)
        assert (off <= room).all(), (self.op, self.shape, (off / room).max())


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("kind", ["bfloat16", "float32"])
def test_exact_sums(gpu, workspace, op, fmt, kind):
    torch = gpu
    for n, size in enumerate(SIZES):
        for space in (None, workspace):
            pad, offset = [(0, 0), (1, 1), (8, 8), (3, 0)][n % 4]
            case = Case(torch, op, *size, fmt, True, n, ("fp4", "fp8")[n % 2], pad, offset)
            flat, out = case.out(getattr(torch, kind), *[(0, 0), (3, 1), (8, 0)][n % 3])
            before = flat.clone()
            case.call(out, space)
            case.check_equal(out)
            out.fill_(55.0)
            assert torch.equal(flat, before)   # nothing written around the output


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_normals(gpu, workspace, op, fmt):
    torch = gpu
    for n, size in enumerate([(1, 300, 700), (19, 257, 130), (140, 200, 333), (300, 384, 512)]):
        for xfmt in ("fp4", "fp8") if op == "product" else ("fp4",):
            case = Case(torch, op, *size, fmt, False, 50 + n, xfmt, n % 2)
            for kind in (torch.bfloat16, torch.float32):
                for space in (None, workspace):
                    _, out = case.out(kind)
                    case.call(out, space)
                    case.check_near(out)


@pytest.mark.parametrize("op,size", [
    ("linear", (1, 100, 20000)), ("linear", (33, 64, 9000)), ("linear", (8, 4096, 1024)),
    ("product", (1, 100, 20000)), ("product", (70, 300, 8192)), ("product", (16, 4096, 2048)),
    ("product", (65, 4096, 8190)), ("product", (70, 200, 2337)), ("product", (33, 500, 4609)),
    ("dgrad", (5, 20000, 70)), ("dgrad", (129, 9000, 130)), ("dgrad", (1, 512, 4096)),
    ("wgrad", (20000, 60, 70)), ("wgrad", (9001, 129, 257)), ("wgrad", (4096, 128, 1024))])
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_long_sums(gpu, workspace, op, size, fmt):
    """Depths that are split over workgroups: still exact, the workspace left ready."""
    torch = gpu
    case = Case(torch, op, *size, fmt, True, 7)
    for space in (None, workspace, workspace):
        for kind in (torch.float32, torch.bfloat16):
            _, out = case.out(kind)
            case.call(out, space)
            case.check_equal(out)
    assert not workspace[:65536].any()


@pytest.mark.parametrize("size", [(1024, 2048, 1024), (2050, 1031, 1090), (515, 4104, 776)])
@pytest.mark.parametrize("op", OPS)
def test_large(gpu, workspace, op, size):
    """Sizes of many tiles, exact sums."""
    torch = gpu
    fmt = "fp8" if op == "wgrad" else "fp4"
    case = Case(torch, op, *size, fmt, True, 11, "fp4", pad=size[0] % 2)
    for kind in (torch.bfloat16, torch.float32):
        _, out = case.out(kind)
        case.call(out, workspace)
        case.check_equal(out)


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_gradient_added(gpu, workspace, fmt):
    torch = gpu
    for size in [(3, 33, 31), (130, 100, 96), (9001, 129, 257)]:
        case = Case(torch, "wgrad", *size, fmt, True, 3, pad=1)
        rng = np.random.default_rng(1)
        old = rng.integers(-1000, 1000, case.shape).astype(np.float32)
        for space in (None, workspace):
            _, out = case.out(torch.float32, 3, 1, old)
            case.call(out, space, add=True)
            case.check_equal(out, old)
            case.call(out, space, add=True)
            case.check_equal(out, old + case.want)


@pytest.mark.parametrize("op", OPS)
def test_empty_sums(gpu, workspace, op):
    """No depth: zeros are written (or nothing added); no outputs: nothing happens."""
    torch = gpu
    sizes = {"linear": (5, 7, 0), "product": (5, 7, 0), "dgrad": (5, 0, 7), "wgrad": (0, 5, 7)}
    case = Case(torch, op, *sizes[op], "fp4", True, 0)
    for space in (None, workspace):
        _, out = case.out(torch.float32)
        case.call(out, space)
        assert not out.any()
        if op == "wgrad":
            out.fill_(3.0)
            case.call(out, space, add=True)
            assert (out == 3.0).all()
    for size in ((0, 7, 64), (5, 0, 64) if op != "dgrad" else (5, 64, 0)):
        if op == "wgrad" and size[0] == 0:
            continue
        case = Case(torch, op, *size, "fp4", True, 0)
        case.call(case.out(torch.float32)[1], workspace)
    torch.cuda.synchronize()


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("size", [(1, 100, 200), (40, 70, 96), (300, 260, 290)])
def test_nonfinite(gpu, workspace, op, size):
    """NaN and infinities reach the sums that hold them, and no other."""
    torch = gpu
    case = Case(torch, op, *size, "fp4", True, 5, "fp8")
    clean = case.want.copy()
    i, c = case.shape[0] // 2, case.depth // 3
    j, d = case.shape[1] // 3, case.depth - 1
    # one infinity in the first operand, one NaN block in the second
    if op == "product":
        case.a.scales[i, c // 32] = 255
    elif op == "wgrad":
        case.a[c, i] = float("inf")
    else:
        case.a[i, c] = float("inf")
    if op in ("linear", "product"):
        case.b.scales[j, d // 32] = 255
        bad = [j]
    else:
        case.b.scales[d, j // 32] = 255
        bad = range(j // 32 * 32, min(j // 32 * 32 + 32, case.shape[1]))
    for kind in (torch.bfloat16, torch.float32):
        _, out = case.out(kind)
        case.call(out, workspace)
        got = out.float().cpu().numpy()
        touched = np.zeros(case.shape, bool)
        touched[i] = True
        touched[:, list(bad)] = True
        assert np.isnan(got[:, list(bad)]).all()
        if op == "product":
            assert np.isnan(got[i]).all()
        else:
            assert not np.isfinite(got[i]).any()
        want = ref.bf16_round(clean) if kind == torch.bfloat16 else clean.astype(np.float32)
        assert np.array_equal(got[~touched], want[~touched])


def test_extreme_scales(gpu):
    """Powers of two at both ends; the sums stay what the exact ones round to."""
    torch = gpu
    for b in (1, 20, 127, 230, 250):
        codes = np.full((40, 16), 0x42, np.uint8)           # 1, 2, 1, 2 ...
        scales = np.full((40, 1), b, np.uint8)
        w = zs.Mx(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), 32, "fp4")
        x = torch.full((3, 32), 2.0 ** (-60 if b > 127 else 60), dtype=torch.bfloat16,
                       device="cuda")
        y = torch.empty(3, 40, device="cuda")
        zs.zs_mx_linear(x, w, y, torch.cuda.current_stream())
        want = 48.0 * 2.0 ** (b - 127) * float(x[0, 0])
        assert (y == want).all(), b


@pytest.mark.parametrize("op", OPS)
def test_same_bits_every_time_and_on_a_stream(gpu, op):
    torch = gpu
    case = Case(torch, op, 70, 3000 if op == "dgrad" else 200, 210 if op == "dgrad" else 3000,
                "fp4", False, 1)
    if op == "wgrad":
        case = Case(torch, op, 5000, 100, 130, "fp8", False, 1)
    space = zs.mx_workspace()
    _, first = case.out(torch.float32)
    case.call(first, space)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        _, out = case.out(torch.float32)
        side.wait_stream(torch.cuda.current_stream())
        case.call(out, space, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, first)


@pytest.mark.parametrize("op", OPS)
def test_captured_and_replayed(gpu, op):
    """A graph of two calls on one workspace, replayed on other inputs between eager work."""
    torch = gpu
    size = {"dgrad": (20, 6000, 100), "wgrad": (6000, 90, 100)}.get(op, (20, 100, 6000))
    cases = [Case(torch, op, *size, "fp8", True, s) for s in range(3)]
    live = Case(torch, op, *size, "fp8", True, 0)
    space = zs.mx_workspace()
    _, out = live.out(torch.float32)
    _, out2 = live.out(torch.bfloat16)
    live.call(out, space)                  # the kernel is loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        live.call(out, space)
        live.call(out2, space)
    for case in cases + cases:
        for to, of in ((live.a, case.a), (live.b, case.b)):
            if isinstance(to, zs.Mx):
                to.codes.copy_(of.codes)
                to.scales.copy_(of.scales)
            else:
                to.copy_(of)
        graph.replay()
        torch.cuda.synchronize()
        case.check_equal(out)
        case.check_equal(out2)
        out.zero_()
        out2.zero_()
        case.call(out, space)              # eager on the same workspace
        case.check_equal(out)
        torch.randn(4096, device="cuda").square().sum().item()


def test_workspace_of_a_capture_is_refused_outside(gpu):
    torch = gpu
    case = Case(torch, "linear", 3, 40, 64, "fp4", True, 0)
    _, out = case.out(torch.float32)
    case.call(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        space = zs.mx_workspace()
        case.call(out, space)
    with pytest.raises(ValueError, match="made during a graph capture"):
        case.call(out, space)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        case.check_equal(out)


def test_linear_gradients_against_differences(gpu):
    """dgrad and wgrad are the derivatives of sum(c * (x w^T)), which is linear in x and in w:
    differences of the exact forward product give them."""
    torch = gpu
    rng = np.random.default_rng(2)
    m, n, k = 6, 10, 40
    x, xv = held(torch, rng, m, k, "fp8", True)
    w, wv = held(torch, rng, n, k, "fp4", True)
    c = torch.from_numpy(rng.integers(-4, 5, (m, n)).astype(float)).to(torch.bfloat16)
    cv = c.double().numpy()

    def loss(xv, wv):
        return (cv * (xv @ wv.T)).sum()

    dx = torch.empty(m, k, device="cuda")
    dw = torch.empty(n, k, device="cuda")
    zs.zs_mx_linear_dgrad(c.cuda(), w, dx, torch.cuda.current_stream())
    zs.zs_mx_linear_wgrad(c.cuda(), x, dw, False, torch.cuda.current_stream())
    for got, at, other, first in ((dx, xv, wv, True), (dw, wv, xv, False)):
        got = got.cpu().numpy()
        for i, j in zip(rng.integers(0, at.shape[0], 12), rng.integers(0, at.shape[1], 12)):
            up, down = at.copy(), at.copy()
            up[i, j] += 1
            down[i, j] -= 1
            diff = (loss(up, other) - loss(down, other)) / 2 if first else \
                (loss(other, up) - loss(other, down)) / 2
            assert got[i, j] == diff


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_aligned_rows(gpu, workspace, op, fmt):
    """Rows a multiple of 16 bytes apart, with and without a rest past the last whole chunk
    (the gaps hold NaN), every number of steps around a turn of the loops."""
    torch = gpu
    for n, depth in enumerate((225, 256, 257, 263, 320, 384, 449, 511, 512, 513, 700, 1031, 1279,
                               2048, 2111)):
        m, other = [(3, 130), (130, 257), (257, 70), (70, 300)][n % 4]
        size = {"dgrad": (m, depth, other), "wgrad": (depth, m, other)}.get(op, (m, other, depth))
        width = m if op == "wgrad" else depth
        case = Case(torch, op, *size, fmt, True, n, ("fp4", "fp8")[n % 2], -width % 8, 8 * (n % 3))
        for space in (None, workspace):
            for kind in (torch.float32, torch.bfloat16):
                _, out = case.out(kind)
                case.call(out, space)
                case.check_equal(out)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
@pytest.mark.parametrize("depth", [320, 1300])
def test_many_tiles(gpu, workspace, op, fmt, depth):
    """Outputs large enough for the largest tiles, ragged at both ends."""
    torch = gpu
    m, other = 4100, 4360
    size = {"dgrad": (m, depth, other), "wgrad": (depth, m, other)}.get(op, (m, other, depth))
    case = Case(torch, op, *size, fmt, True, depth, fmt, 4 if op == "wgrad" else 4 * (depth % 8))
    for kind in (torch.float32, torch.bfloat16):
        flat, out = case.out(kind, 8)
        before = flat.clone()
        case.call(out, workspace)
        case.check_equal(out)
        out.fill_(55.0)
        assert torch.equal(flat, before)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 7, 8, 9])
@pytest.mark.parametrize("pad", [0, 1])
def test_narrow_gradients(gpu, workspace, n, pad):
    """dw of a few rows: dy's rows are shorter than a chunk."""
    torch = gpu
    for m, k in ((1, 40), (64, 33), (65, 100), (130, 64), (9001, 70)):
        case = Case(torch, "wgrad", m, n, k, "fp8", True, m, pad=pad)
        for space in (None, workspace):
            _, out = case.out(torch.float32)
            case.call(out, space)
            case.check_equal(out)


@pytest.mark.parametrize("op", ["linear", "product", "dgrad", "wgrad"])
@pytest.mark.parametrize("pad", [0, 1])
def test_offsets_past_32_bits(gpu, workspace, op, pad):
    """Operands and outputs of more than 2^31 elements or 2^32 bytes: zeros but for a few rows
    near the end, whose products arrive where they belong."""
    torch = gpu
    rows, n, k = 2_100_007, 72, 1056
    rng = np.random.default_rng(4)
    last = torch.tensor([rows - 70, rows - 2, rows - 1])
    w, wv = held(torch, rng, n, k, "fp4", True)
    if op in ("linear", "product"):
        x, xv = plain(torch, rng, 3, k, True, 0, 0)
        y = torch.full((rows, n), 7.0, device="cuda")
        if op == "linear":
            full = torch.zeros(rows, k + pad, dtype=torch.bfloat16, device="cuda")[:, :k]
            full[last.cuda()] = x
            zs.zs_mx_linear(full, w, y, torch.cuda.current_stream(), workspace)
            want = xv @ wv.T
        else:
            full, few = zs.Mx.empty(rows, k, "fp8"), zs.Mx.empty(3, k, "fp8")
            zs.zs_mx_quantize(x, few, torch.cuda.current_stream())
            full.codes.zero_()
            full.scales.fill_(127)
            full.codes[last.cuda()] = few.codes
            full.scales[last.cuda()] = few.scales
            zs.zs_mx_product(full, w, y, torch.cuda.current_stream(), workspace)
            want = ref.decode(few.codes.cpu().numpy(), few.scales.cpu().numpy(), "fp8", k) @ wv.T
        assert np.array_equal(y[last.cuda()].cpu().numpy(), want.astype(np.float32))
        assert int((y != 0).any(1).sum()) == 3
    elif op == "dgrad":
        dy, dv = plain(torch, rng, 3, n, True, 0, 0)
        full = torch.zeros(rows, n + 8 * pad + pad, dtype=torch.bfloat16, device="cuda")[:, :n]
        full[last.cuda()] = dy
        dx = torch.full((rows, k), 7.0, dtype=torch.bfloat16, device="cuda")
        zs.zs_mx_linear_dgrad(full, w, dx, torch.cuda.current_stream(), workspace)
        assert np.array_equal(dx[last.cuda()].float().cpu().numpy(), ref.bf16_round(dv @ wv))
        assert int((dx != 0).any(1).sum()) == 3
    else:
        dy, dv = plain(torch, rng, 3, n, True, 0, 0)
        few, fv = held(torch, rng, 3, k, "fp8", True)
        full = torch.zeros(rows, n + pad, dtype=torch.bfloat16, device="cuda")[:, :n]
        full[last.cuda()] = dy
        x = zs.Mx.empty(rows, k, "fp8")
        x.codes.fill_(0x38)                          # ones, against zeros of dy
        x.scales.fill_(127)
        x.codes[last.cuda()] = few.codes
        x.scales[last.cuda()] = few.scales
        dw = torch.empty(n, k, device="cuda")
        zs.zs_mx_linear_wgrad(full, x, dw, False, torch.cuda.current_stream(), workspace)
        assert np.array_equal(dw.cpu().numpy(), (dv.T @ fv).astype(np.float32))


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("spread", [10, 60])
def test_scales_far_apart(gpu, workspace, op, spread):
    """Blocks whose powers of two differ by up to 2^120 in one sum: within the same bound."""
    torch = gpu
    size = {"wgrad": (500, 90, 100), "dgrad": (90, 500, 100)}.get(op, (90, 100, 500))
    case = Case(torch, op, *size, "fp4", False, 8)
    rng = np.random.default_rng(9)
    for mx in (case.a, case.b):
        if isinstance(mx, zs.Mx):
            s = rng.integers(127 - spread, 128 + spread, tuple(mx.scales.shape)).astype(np.uint8)
            mx.scales.copy_(torch.from_numpy(s))

    def value(x):
        return ref.decode(x.codes.cpu().numpy(), x.scales.cpu().numpy(), x.format, x.cols) \
            if isinstance(x, zs.Mx) else x.double().cpu().numpy()

    a, b = value(case.a), value(case.b)
    a, b = (a.T if op == "wgrad" else a), (b if op in ("dgrad", "wgrad") else b.T)
    case.want, case.sizes = a @ b, np.abs(a) @ np.abs(b)
    for kind in (torch.float32, torch.bfloat16):
        for space in (None, workspace):
            _, out = case.out(kind)
            case.call(out, space)
            case.check_near(out)
