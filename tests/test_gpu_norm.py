"""The global gradient norm, the scaling of lists of tensors by its coefficient
and the clipping rule on the GPU, against plain implementations in 64 bits.

Tolerances.  The reduced gradient is formed in binary32 in the step's order on
both sides, so the squares are of the same numbers.  The library adds n squares
in binary64: each product and each addition is off by at most 2^-53 of terms
that are all positive, so S is within n 2^-53 of the exact sum (relative), and
norm = sqrt(S) within half of that, plus 2^-53, plus half a step of binary32
(2^-24) for its one rounding; coef = max_norm / (norm + eps) has the same
bound.  n <= 2^32 here: 2^-21 in the worst order, but a lane's own chain and
a tree are at most n / 2^14 + 2^14 additions deep on any of these grids, so
REL = 2^-24 + 2^-34 covers every case.  Scaled tensors are one binary32 product
and one rounding: equal bit for bit to the same on the host."""
import math

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs

pytestmark = pytest.mark.gpu

REL = 2.0 ** -24 + 2.0 ** -34
F32_MAX = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def gpu():
    import torch
    assert torch.cuda.is_available()
    torch.cuda.set_device(0)
    rc = zs.zs_init(0)
    assert rc == zs.ZS_OK, zs.zs_status_string(rc)
    yield torch
    torch.cuda.synchronize()


def bf16_bits(x):
    """bf16 patterns of the values cut to 16 bits."""
    return (np.asarray(x, np.float32).view(np.uint32) >> 16).astype(np.uint16)


def widen(bits):
    return (bits.astype(np.uint32) << 16).view(np.float32)


def fold(values, grad_scale):
    """Left fold in binary32, then the scale."""
    with np.errstate(all="ignore"):
        g = values[0].astype(np.float32)
        for v in values[1:]:
            g = g + v
        return g * np.float32(grad_scale)


def reference(g, max_norm=math.inf, eps=0.0):
    """(S, norm, coef) of the elements in 64 bits."""
    x = np.asarray(g, np.float64).reshape(-1)
    s = math.fsum((x * x).tolist()) if np.isfinite(x).all() else float(np.sum(x * x))
    return (s,) + rule_of(s, max_norm, eps)


def rule_of(s, max_norm, eps):
    norm = math.sqrt(s) if s == s else math.nan
    d = norm + eps
    return norm, (1.0 if d <= max_norm else max_norm / d if d == d else math.nan)


def close(got, want, rel=REL):
    if math.isnan(want):
        return math.isnan(got)
    if want > F32_MAX * (1 + 2.0 ** -25):
        return got == math.inf
    # an fp32 below the normal range is off by half its step, 2^-150
    return abs(got - want) <= rel * abs(want) + 2.0 ** -150


def check(rec, s, norm, coef, apply=1):
    got = rec.sumsq.item(), rec.norm.item(), rec.coef.item(), rec.apply.item()
    want = (s, norm, coef, apply)
    assert math.isnan(s) == math.isnan(got[0]), (got, want)
    if math.isfinite(s):
        assert abs(got[0] - s) <= 2.0 ** -34 * s, (got, want)
    elif not math.isnan(s):
        assert got[0] == s, (got, want)
    assert close(got[1], norm) and close(got[2], coef) and got[3] == apply, (got, want)


def on_gpu(torch, bits, guard=0x7fc0):
    """bf16 patterns on the GPU, with NaN behind the last one."""
    room = np.full(len(bits) + 64, guard, np.uint16)
    room[:len(bits)] = bits
    return torch.from_numpy(room.view(np.int16)).cuda()


def partials(rng, n, k, sigma=1e-2):
    return [bf16_bits(rng.normal(0, sigma, n)) for _ in range(k)]


def norm_of(torch, parts, n, rule=None, grad_scale=1.0, scales=None, stream=None):
    rec = zs.ClipRecord()
    rec.buffer.fill_(0xA5)
    zs.GradNorm(parts, n, rule, rec, grad_scale, scales)(
        torch.cuda.current_stream() if stream is None else stream)
    return rec


SIZES = [1, 2, 3, 7, 8, 9, 15, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1023, 1025, 2047, 2049,
         4095, 4097, 16385, 100003, (1 << 20) + 5]


@pytest.mark.parametrize("k", [1, 2, 3, 4, 7, 8, 16])
def test_norm_of_bf16_partials(gpu, k):
    rng = np.random.default_rng(k)
    for n in SIZES:
        bits = partials(rng, n, k)
        scale = float(rng.choice([1.0, 0.125, 0.3]))
        g = fold([widen(b) for b in bits], scale)
        for max_norm in (math.inf, 0.37 * float(np.linalg.norm(g.astype(np.float64)))):
            rule = zs.clip_rule(max_norm, 1e-6)
            rec = norm_of(gpu, [on_gpu(gpu, b) for b in bits], n, rule, scale)
            check(rec, *reference(g, float(rule.max_norm), float(rule.eps)))


@pytest.mark.parametrize("k", list(range(1, 17)))
def test_norm_of_int8_partials_and_every_count(gpu, k):
    rng = np.random.default_rng(100 + k)
    for n in (1, 5, 16, 17, 255, 256, 257, 1000, 4099, 70001):
        nb = -(-n // 256)
        codes = [rng.integers(-127, 128, n).astype(np.int8) for _ in range(k)]
        scales = [rng.uniform(1e-5, 1e-3, nb).astype(np.float32) for _ in range(k)]
        g = fold([c.astype(np.float32) * np.repeat(s, 256)[:n] for c, s in zip(codes, scales)],
                 0.25)
        pad = [np.concatenate([c, np.full(64, 127, np.int8)]) for c in codes]
        nan = [np.concatenate([s, np.full(16, np.nan, np.float32)]) for s in scales]
        rec = norm_of(gpu, [gpu.from_numpy(c).cuda() for c in pad], n, zs.clip_rule(0.01), 0.25,
                      [gpu.from_numpy(s).cuda() for s in nan])
        check(rec, *reference(g, float(np.float32(0.01)), float(np.float32(1e-6))))
        bits = partials(rng, n, k)
        rec = norm_of(gpu, [on_gpu(gpu, b) for b in bits], n, None, 2.0)
        check(rec, *reference(fold([widen(b) for b in bits], 2.0)))


def test_norm_of_nothing(gpu):
    rec = zs.ClipRecord()
    rec.buffer.fill_(0xA5)
    zs.zs_grad_norm([None], 1, 0, 1.0, zs.clip_rule(1.0), rec, zs.norm_workspace())
    check(rec, 0.0, 0.0, 1.0)
    # max_norm 0 clips everything but a norm of 0
    zs.zs_grad_norm([None], 1, 0, 1.0, zs.clip_rule(0.0, 0.0), rec, zs.norm_workspace())
    check(rec, 0.0, 0.0, 1.0)
    rec = norm_of(gpu, [on_gpu(gpu, bf16_bits([3.0, 4.0]))], 2, zs.clip_rule(0.0))
    check(rec, 25.0, 5.0, 0.0)


def test_range_of_the_squares(gpu):
    """Squares far outside binary32's range, and norms at both of its ends."""
    rule = zs.clip_rule(1.0, 0.0)
    for values in ([2.0 ** 127] * 5, [2.0 ** -130] * 700, [2.0 ** -133], [2.0 ** 127, 2.0 ** -100],
                   [3e38], [3e38, 3e38], [1e-30] * 999 + [1e20], [0.0] * 300 + [2.0 ** -126]):
        bits = bf16_bits(np.array(values, np.float32))
        rec = norm_of(gpu, [on_gpu(gpu, bits)], len(values), rule)
        check(rec, *reference(widen(bits), 1.0, 0.0))


@pytest.mark.parametrize("n", [1, 9, 300, 4099, 100003])
def test_infinities_and_nan(gpu, n):
    rng = np.random.default_rng(n)
    for at in sorted({0, n // 2, n - 1}):
        for bad, s in ((0x7f80, math.inf), (0xff80, math.inf), (0x7fc0, math.nan),
                       (0xffc1, math.nan)):
            bits = partials(rng, n, 2)
            bits[1][at] = bad
            parts = [on_gpu(gpu, b) for b in bits]
            check(norm_of(gpu, parts, n, zs.clip_rule(1.0)), s, s, 0.0 if s == s else math.nan)
            check(norm_of(gpu, parts, n, zs.clip_rule(1.0, skip_nonfinite=True)), s, s,
                  0.0 if s == s else math.nan, 0)
            check(norm_of(gpu, parts, n), s, s, 1.0 if s == s else math.nan)
    # opposite infinities in the two partials: their sum is NaN
    bits = partials(rng, n, 2)
    bits[0][n - 1], bits[1][n - 1] = 0x7f80, 0xff80
    check(norm_of(gpu, [on_gpu(gpu, b) for b in bits], n, zs.clip_rule(1.0)), math.nan, math.nan,
          math.nan)


def test_elements_past_32_bits(gpu):
    """A shard of more than 2^31 elements (and 2^32 bytes): zeros but for a few
    elements around the places where an index could wrap."""
    torch, n = gpu, (1 << 31) + 4097
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = [0, 1, (1 << 30) + 3, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 2, n - 1]
    for j, i in enumerate(at):
        g[i] = float(1 << j)
    s = float(sum(4 ** j for j in range(len(at))))
    rec = norm_of(torch, [g], n, zs.clip_rule(2.0, 0.0))
    check(rec, s, math.sqrt(s), 2.0 / math.sqrt(s))


@pytest.mark.parametrize("k,form", [(1, "bf16"), (2, "bf16"), (3, "bf16"), (8, "bf16"),
                                    (1, "int8"), (2, "int8"), (9, "int8")])
def test_every_element_of_a_large_shard_counts_once(gpu, k, form):
    """Shards on both sides of 2^26 elements and of 4 MB of partials, where the order
    of the work changes, with ragged numbers of tiles: all ones, so that S = n k^2 exactly."""
    torch = gpu
    top = (1 << 26) + 8 * 70001 + 5
    if form == "int8":
        parts = [torch.ones(top, dtype=torch.int8, device="cuda")] * k
        scales = [torch.ones(-(-top // 256), device="cuda")] * k
    else:
        parts, scales = [torch.ones(top, dtype=torch.bfloat16, device="cuda")] * k, None
    for n in (1 << 18, (1 << 19) - 1, 1 << 19, 524_289 + 777, 1 << 24, (1 << 26) - 1, 1 << 26,
              (1 << 26) + 1, (1 << 26) + 4097, top):
        rec = norm_of(torch, parts, n, None, 1.0, scales)
        assert rec.sumsq.item() == float(n * k * k), n


@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
def test_every_element_of_a_large_list_counts_and_is_scaled_once(gpu, dtype):
    torch = gpu
    sizes = [60_000_001, 1, 8191, 70_000_003, 3, 4096, 20_000_000]
    flat = torch.ones(sum(sizes), dtype=getattr(torch, dtype), device="cuda")
    table, rec = zs.TensorTable(flat.split(sizes)), zs.ClipRecord()
    zs.TensorsNorm(table, zs.clip_rule(0.5 * math.sqrt(sum(sizes)), 0.0), rec)()
    assert rec.sumsq.item() == float(sum(sizes)) and abs(rec.coef.item() - 0.5) <= 2.0 ** -25
    zs.zs_tensors_clip(table, rec)
    assert bool((flat == (torch.ones(1) * rec.coef.cpu()).to(flat.dtype).cuda()).all())


def test_many_calls_on_one_workspace(gpu):
    """The arrival counters are back at 0 after every call: grids of one, a few,
    tens, hundreds and a thousand workgroups in turn on one workspace."""
    torch = gpu
    rng = np.random.default_rng(77)
    ws = zs.norm_workspace()
    calls = []
    for n in (5, 9000, 300_000, 40_000, 4_000_000, 2_000, 16_000_000, 140_000):
        b = bf16_bits(np.ones(n) * float(rng.integers(1, 9)))
        rec = zs.ClipRecord()
        calls.append((zs.GradNorm([on_gpu(torch, b)], n, None, rec, workspace=ws), rec,
                      n * float(widen(b)[0]) ** 2))
    for rep in range(40):
        for j in rng.permutation(len(calls)):
            calls[j][0]()
        torch.cuda.synchronize()
        for _, rec, s in calls:
            assert rec.sumsq.item() == s
            rec.buffer.zero_()
    assert not ws[:64].any()


def test_same_call_same_bits(gpu):
    torch, n = gpu, 5_000_011
    rng = np.random.default_rng(5)
    parts = [on_gpu(torch, b) for b in partials(rng, n, 3)]
    first = norm_of(torch, parts, n, zs.clip_rule(1.0)).buffer
    for _ in range(5):
        assert torch.equal(norm_of(torch, parts, n, zs.clip_rule(1.0)).buffer, first)


def test_combine(gpu):
    torch = gpu
    rng = np.random.default_rng(9)
    for count in (1, 2, 8, 63, 256, 257, 1000, zs.ZS_MAX_SUMS):
        sums = rng.uniform(0, 3, count)
        rec = zs.ClipRecord()
        dev = torch.from_numpy(np.append(sums, np.nan)).cuda()[:count]
        zs.zs_clip_combine(dev, zs.clip_rule(1.5, 0.25), rec)
        s = math.fsum(sums.tolist())
        check(rec, s, *rule_of(s, 1.5, 0.25))
    # the record's own sum after the other ranks' were added to it
    rec.sumsq.fill_(49.0)
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(3.5, 0.0), rec)
    check(rec, 49.0, 7.0, 0.5)
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(7.0, 0.0), rec)   # the norm at the border
    check(rec, 49.0, 7.0, 1.0)
    rec.sumsq.fill_(math.inf)
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(7.0, 0.0, True), rec)
    check(rec, math.inf, math.inf, 0.0, 0)


DTYPES = ("bfloat16", "float16", "float32")


def lay_out(torch, rng, sizes, dtypes, gaps, special=False):
    """Tensors cut from one buffer per type, with gaps of NaN between them.
    Returns the tensors, the buffers and a mask of the gaps."""
    out, buffers = [None] * len(sizes), []
    for name in DTYPES:
        mine = [i for i in range(len(sizes)) if dtypes[i] == name]
        total = sum(sizes[i] + gaps[i] for i in mine) + 64
        buf = torch.full((total,), math.nan, dtype=getattr(torch, name))
        at = 0
        for i in mine:
            at += gaps[i]
            x = torch.from_numpy(rng.normal(0, 1, sizes[i]))
            if special and sizes[i] > 8:
                x[1], x[3], x[4], x[5] = 0.0, -0.0, 1e-7, 6e4
            buf[at:at + sizes[i]] = x.to(buf.dtype)
            out[i] = (at, sizes[i])
            at += sizes[i]
        dev = buf.cuda()
        for i in mine:
            out[i] = dev[out[i][0]:out[i][0] + out[i][1]]
        buffers.append(dev)
    return out, buffers


def case(torch, seed, count, high):
    rng = np.random.default_rng(seed)
    sizes = [int(rng.choice([0, 1, 2, 3, 7, 8, 9, 63, 64, 65, 511, 513, 4095, 4096, 4097,
                             int(rng.integers(1, high))])) for _ in range(count)]
    dtypes = [str(rng.choice(DTYPES)) for _ in range(count)]
    gaps = [int(rng.integers(0, 9)) for _ in range(count)]
    return lay_out(torch, rng, sizes, dtypes, gaps, special=True)


LISTS = [(1, 1, 10), (2, 5, 100), (3, 40, 5000), (4, 300, 20000), (5, 3, 3_000_000),
         (6, 2000, 300)]


@pytest.mark.parametrize("seed,count,high", LISTS)
def test_norm_and_scaling_of_tensors(gpu, seed, count, high):
    torch = gpu
    tensors, buffers = case(torch, seed, count, high)
    before = [b.clone() for b in buffers]
    values = torch.cat([t.double() for t in tensors]).cpu().numpy() if tensors else np.zeros(0)
    s, norm, _ = reference(values)
    rule = zs.clip_rule(0.3 * norm if norm else 1.0, 1e-6)
    table, rec = zs.TensorTable(tensors), zs.ClipRecord()
    zs.TensorsNorm(table, rule, rec)()
    check(rec, s, *rule_of(s, float(rule.max_norm), float(rule.eps)))
    for a, b in zip(buffers, before):   # the norm reads only
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    zs.zs_tensors_clip(table, rec)
    coef = rec.coef.cpu()
    starts = {(b.dtype, t.data_ptr()) for t in tensors for b in buffers if t.dtype == b.dtype}
    assert starts
    for dev, old in zip(buffers, before):
        old, inside = old.cpu(), torch.zeros(old.numel(), dtype=torch.bool)
        for t in tensors:
            if t.dtype == dev.dtype and t.numel():
                at = (t.data_ptr() - dev.data_ptr()) // dev.element_size()
                inside[at:at + t.numel()] = True
        want = torch.where(inside, (old.float() * coef).to(old.dtype), old)
        got = dev.cpu()
        # the gaps keep their NaN, bit for bit; inside there is none
        kind = torch.int32 if dev.element_size() == 4 else torch.int16
        assert torch.equal(got.view(kind), want.view(kind))


def test_scaling_keeps_signs_infinities_and_nan(gpu):
    torch = gpu
    odd = [math.inf, -math.inf, math.nan, -0.0, 0.0, 1.0, -3.0, 65504.0, 6e-8, 1e-40, 3e38]
    rec = zs.ClipRecord()
    rec.sumsq.fill_(100.0)
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(3.0, 0.0), rec)
    coef = rec.coef.cpu()
    for name in DTYPES:
        for shift in range(9):
            x = torch.tensor(odd * 9, dtype=torch.float32).to(getattr(torch, name))
            dev = torch.zeros(shift + len(x) + 9, dtype=x.dtype, device="cuda")
            dev[shift:shift + len(x)] = x.cuda()
            zs.zs_tensors_clip(zs.TensorTable([dev[shift:shift + len(x)]]), rec)
            want = (x.float() * coef).to(x.dtype)
            got = dev[shift:shift + len(x)].cpu()
            kind = torch.int32 if x.element_size() == 4 else torch.int16
            nan = want.isnan()
            assert torch.equal(got.isnan(), nan)
            assert torch.equal(got.view(kind)[~nan], want.view(kind)[~nan]), (name, shift)
            if name == "bfloat16":
                assert bool((got.view(kind)[nan] == 0x7fc0).all())
            assert not dev[:shift].any() and not dev[shift + len(x):].any()


def test_nothing_is_scaled_without_need(gpu):
    """apply 0 (a record no norm call has written, or a skipped step) and coef 1
    leave every bit, NaN payloads included."""
    torch = gpu
    x = torch.randn(10001, device="cuda")
    x[77] = math.nan
    before = x.clone()
    table = zs.TensorTable([x])
    rec = zs.ClipRecord()
    zs.zs_tensors_clip(table, rec)
    assert torch.equal(x.view(torch.int32), before.view(torch.int32))
    zs.TensorsNorm(table, zs.clip_rule(1.0, skip_nonfinite=True), rec)()
    zs.zs_tensors_clip(table, rec)
    check(rec, math.nan, math.nan, math.nan, 0)
    assert torch.equal(x.view(torch.int32), before.view(torch.int32))
    x[77] = 1.0
    before = x.clone()
    zs.TensorsNorm(table, zs.clip_rule(1e9), rec)()
    zs.zs_tensors_clip(table, rec)
    assert rec.coef.item() == 1.0 and torch.equal(x, before)


def test_tables_of_no_elements(gpu):
    torch = gpu
    for tensors in ([], [torch.zeros(0, device="cuda")]):
        table, rec = zs.TensorTable(tensors), zs.ClipRecord()
        zs.TensorsNorm(table, zs.clip_rule(1.0), rec)()
        check(rec, 0.0, 0.0, 1.0)
        zs.zs_tensors_clip(table, rec)


def test_transposed_and_permuted_tensors(gpu):
    torch = gpu
    a = torch.randn(37, 501, device="cuda").t()
    b = torch.randn(4, 6, 10, dtype=torch.float32, device="cuda").to(torch.bfloat16).permute(2, 0, 1)
    want = [x.clone() for x in (a, b)]
    table, rec = zs.TensorTable([a, b]), zs.ClipRecord()
    zs.TensorsNorm(table, zs.clip_rule(2.0), rec)()
    s, norm, coef = reference(torch.cat([x.double().reshape(-1) for x in want]).cpu().numpy(), 2.0,
                              float(np.float32(1e-6)))
    check(rec, s, norm, coef)
    zs.zs_tensors_clip(table, rec)
    for x, w in zip((a, b), want):
        assert torch.equal(x, (w.float() * rec.coef).to(w.dtype))


def test_a_tensor_of_more_than_4_gib(gpu):
    torch, n = gpu, (1 << 30) + 1029
    x = torch.zeros(n, device="cuda")
    at = [0, 1, (1 << 29) + 1, (1 << 30) - 1, 1 << 30, n - 1]
    for j, i in enumerate(at):
        x[i] = float(3 << j)
    s = float(sum((3 << j) ** 2 for j in range(len(at))))
    table, rec = zs.TensorTable([x]), zs.ClipRecord()
    zs.TensorsNorm(table, zs.clip_rule(1.0, 0.0), rec)()
    check(rec, s, math.sqrt(s), 1.0 / math.sqrt(s))
    zs.zs_tensors_clip(table, rec)
    coef = rec.coef.cpu()
    assert int((x != 0).sum()) == len(at)
    for j, i in enumerate(at):
        assert x[i].cpu() == torch.tensor(float(3 << j)) * coef


def test_replayed_graphs_and_streams(gpu):
    """Norm, combine and scaling captured into one graph and replayed on new
    values, with eager work in between; then two streams at once, each with a
    workspace and a record of its own."""
    torch = gpu
    rng = np.random.default_rng(31)
    n, rule = 300_007, zs.clip_rule(1.0)
    grad = on_gpu(torch, partials(rng, n, 1)[0])
    rest = [torch.randn(999, device="cuda"), torch.randn(4100, device="cuda").half()]
    rec, rec2 = zs.ClipRecord(), zs.ClipRecord()
    sums = torch.zeros(2, dtype=torch.float64, device="cuda")
    table = zs.TensorTable(rest)
    norm, norm2 = zs.GradNorm([grad], n, None, rec), zs.TensorsNorm(table, None, rec2)

    def whole(stream):
        norm(stream)
        norm2(stream)
        sums[0:1].copy_(rec.sumsq)
        sums[1:2].copy_(rec2.sumsq)
        zs.zs_clip_combine(sums, rule, rec, stream)
        zs.zs_tensors_clip(table, rec, stream)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        whole(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for rep in range(4):
        bits = partials(rng, n, 1, 10.0 ** -rep)[0]
        grad[:n] = torch.from_numpy(bits.view(np.int16)).cuda()
        new = [torch.from_numpy(rng.normal(0, 1, t.numel())).to(t.dtype) for t in rest]
        for t, x in zip(rest, new):
            t.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        s = reference(np.concatenate([widen(bits).astype(np.float64)] +
                                     [x.double().numpy() for x in new]))[0]
        check(rec, s, *rule_of(s, 1.0, float(np.float32(1e-6))))
        for t, x in zip(rest, new):
            assert torch.equal(t.cpu(), (x.float() * rec.coef.cpu()).to(x.dtype))
        got = [rec.buffer.clone(), *(t.clone() for t in rest)]
        for t, x in zip(rest, new):
            t.copy_(x)
        whole(torch.cuda.current_stream())     # the same eagerly
        torch.cuda.synchronize()
        for a, b in zip(got, [rec.buffer, *rest]):
            assert torch.equal(a, b)

    streams = [torch.cuda.Stream() for _ in range(2)]
    bits = [partials(rng, n, 2) for _ in streams]
    parts = [[on_gpu(torch, b) for b in bs] for bs in bits]
    recs = [zs.ClipRecord() for _ in streams]
    calls = [zs.GradNorm(p, n, rule, r) for p, r in zip(parts, recs)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, st in zip(calls, streams):
            c(st)
    torch.cuda.synchronize()
    for bs, r in zip(bits, recs):
        check(r, *reference(fold([widen(b) for b in bs], 1.0), 1.0, float(np.float32(1e-6))))


def test_objects_made_on_a_busy_stream_are_ready_on_another(gpu):
    """Record, workspace and table are made while the current stream is busy, and
    used at once on another stream."""
    torch = gpu
    side, n = torch.cuda.Stream(), 700_001
    bits = partials(np.random.default_rng(8), n, 1)
    part = on_gpu(torch, bits[0])
    x = torch.ones(300_000, device="cuda")
    garbage = torch.full((1 << 20,), 0x55, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    del garbage                            # what a new allocation may find in its memory
    for rep in range(4):
        torch.cuda._sleep(20_000_000)
        rec, rec_x = zs.ClipRecord(), zs.ClipRecord()
        norm = zs.GradNorm([part], n, zs.clip_rule(1.0), rec)
        norm_x = zs.TensorsNorm(zs.TensorTable([x]), zs.clip_rule(1.0), rec_x)
        norm(side)
        norm_x(side)
        side.synchronize()
        check(rec, *reference(widen(bits[0]), 1.0, float(np.float32(1e-6))))
        assert rec_x.sumsq.item() == 300_000.0
    torch.cuda.synchronize()


def test_objects_made_during_a_capture(gpu):
    """Their zeroing becomes part of the graph: every replay starts from it."""
    torch, n = gpu, 500_009
    rng = np.random.default_rng(12)
    part = on_gpu(torch, partials(rng, n, 1)[0])
    norm_of(torch, [part], n)              # the kernel is loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec = zs.ClipRecord()
        norm = zs.GradNorm([part], n, zs.clip_rule(1.0), rec)
        norm(torch.cuda.current_stream())
    for _ in range(4):
        bits = partials(rng, n, 1)[0]
        part[:n] = torch.from_numpy(bits.view(np.int16)).cuda()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check(rec, *reference(widen(bits), 1.0, float(np.float32(1e-6))))
        assert torch.isfinite(torch.randn(4096, device="cuda").square().sum())
        torch.cuda.synchronize()


def test_errors_are_reported(gpu):
    rec, ws = zs.ClipRecord(), zs.norm_workspace()
    g = on_gpu(gpu, np.zeros(64, np.uint16))
    with pytest.raises(zs.ZsError, match="invalid argument"):
        zs.zs_grad_norm([g], 1, 64, math.nan, None, rec, ws)
    with pytest.raises(TypeError, match=r"grads\[0\] is torch.float16"):
        zs.zs_grad_norm([g.view(gpu.float16)], 1, 64, 1.0, None, rec, ws)
    with pytest.raises(TypeError, match=r"qscales\[0\] is torch.int32"):
        zs.zs_grad_norm_q8grad([g.view(gpu.int8)], [g.view(gpu.int32)], 1, 64, 1.0, None, rec, ws)
    with pytest.raises(zs.ZsError, match="not aligned"):
        zs.zs_grad_norm([g[1:]], 1, 8, 1.0, None, rec, ws)
    with pytest.raises(zs.ZsError, match="overlap"):
        zs.zs_grad_norm([ws.view(gpu.int16)], 1, 64, 1.0, None, rec, ws)
    assert zs.zs_clip_combine(rec.sumsq, zs.clip_rule(-1.0), rec, check=False) == \
        zs.ZS_ERR_INVALID_ARGUMENT
    assert rec.apply.item() == 0     # nothing was enqueued
