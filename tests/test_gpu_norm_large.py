"""Norm, scaling and clipped step at sizes above one round of workgroups, across
the borders where the order, the kind of loads and the occupancy change, on
random data made on the GPU: every tile's sum of squares is its own, so a tile
read twice in another's place shows.

Tolerance.  S of n elements: each side adds squares of the same binary32 numbers
in binary64, all positive, within (depth of its additions) x 2^-53.  A lane of the
library adds at most n / 2^17 < 2^13 elements (512 workgroups of 256 lanes or more),
then come a few hundred lanes' and workgroups' sums; torch's stretches of 2^22
elements are summed over thousands of lanes, at most 2^12 deep, then on the host
exactly: 2^-53 (2^13 + 2^12 + 2^10) < 2^-39.  A tile of at least 2^14 elements
swapped for another changes S by about 2^-7 of one of at most 2^16 tiles: 2^-23."""
import math

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _gpu_harness as H
from tests.test_gpu_clipped_step import hp_of
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

SUM_REL = 2.0 ** -39
COUNTER_BYTES = 33 * 128     # one counter and 32 of the second level, a cache line each
STRETCH = 1 << 22


def gradient(torch, parts, scales, a, b, grad_scale):
    """Elements a .. b - 1 of the reduced gradient, binary32, in the step's order."""
    g = None
    for j, p in enumerate(parts):
        x = p[a:b].float()
        if scales is not None:     # a is a multiple of a block
            x *= scales[j][a // 256:-(-b // 256)].repeat_interleave(256)[:b - a]
        g = x if g is None else g + x
    return g * grad_scale


def sum_of_squares(torch, parts, scales, n, grad_scale):
    sums = []
    for a in range(0, n, STRETCH):
        g = gradient(torch, parts, scales, a, min(n, a + STRETCH), grad_scale).double()
        sums.append((g * g).sum())
    return math.fsum(torch.stack(sums).cpu().tolist())


def partials(torch, form, n, k, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    room = n + 40                # what lies behind must not count
    if form == "int8":
        parts = [torch.empty(room, dtype=torch.int8, device="cuda").random_(-127, 128, generator=gen)
                 for _ in range(k)]
        scales = [torch.rand(-(-n // 256), device="cuda", generator=gen).mul_(1e-4) for _ in range(k)]
        return parts, scales
    return [torch.empty(room, dtype=torch.bfloat16, device="cuda").normal_(0, 1e-2, generator=gen)
            for _ in range(k)], None


# around 2^26 elements, 4 MB of partials and 256 MB of partials, ragged
@pytest.mark.parametrize("form,n,k", [
    ("bf16", (1 << 26) - 5, 1), ("bf16", (1 << 26) + 4099, 1), ("bf16", 300_000_007, 1),
    ("bf16", 150_000_003, 2), ("bf16", 20_000_001, 3), ("bf16", 700_001, 4),
    ("bf16", 60_000_011, 4), ("bf16", 31_000_001, 5), ("bf16", 90_000_013, 7),
    ("bf16", 80_000_009, 8), ("bf16", 21_000_005, 16), ("int8", 600_000_019, 1),
    ("int8", 200_000_029, 2), ("int8", 66_000_007, 5), ("int8", 35_000_001, 8),
    ("int8", 70_000_003, 9), ("int8", 17_000_023, 16)])
def test_norm_of_random_partials(gpu, form, n, k):
    torch = gpu
    parts, scales = partials(torch, form, n, k, n % 1000 + k)
    ws = zs.norm_workspace()
    for grad_scale in (1.0, 0.3):
        rec = zs.ClipRecord()
        zs.GradNorm(parts, n, zs.clip_rule(1.0), rec, grad_scale, scales, ws)()
        want = sum_of_squares(torch, parts, scales, n, grad_scale)
        got = rec.sumsq.item()
        assert abs(got - want) <= SUM_REL * want, (got / want - 1, grad_scale)
        # every arrival counter is back at 0, those of the second level, too
        assert not ws[:COUNTER_BYTES].any()


@pytest.mark.parametrize("dtypes,count,total", [
    (("bfloat16",), 97, 300_000_011), (("float32",), 11, 90_000_001), (("float16",), 203, 40_000_003),
    (("bfloat16", "float32", "float16"), 301, 250_000_037)])
def test_norm_and_scaling_of_random_lists(gpu, dtypes, count, total):
    torch = gpu
    rng = np.random.default_rng(total)
    share = rng.uniform(0.1, 1.0, count) * np.where(np.arange(count) % 3 == 0, 1e-3, 1.0)
    sizes = [max(1, int(x)) for x in share / share.sum() * total]
    buffers, tensors, inside = [], [], []
    for j, name in enumerate(dtypes):
        mine = [s for i, s in enumerate(sizes) if i % len(dtypes) == j]
        gaps = [int(rng.integers(0, 9)) for _ in mine]
        buf = torch.randn(sum(mine) + sum(gaps) + 16, device="cuda").to(getattr(torch, name))
        mask = torch.zeros(buf.numel(), dtype=torch.bool, device="cuda")
        at = 0
        for s, gap in zip(mine, gaps):
            at += gap
            tensors.append(buf[at:at + s])
            mask[at:at + s] = True
            at += s
        buffers.append(buf)
        inside.append(mask)
    before = [b.clone() for b in buffers]
    want = math.fsum(float((p.double() ** 2).sum()) for t in tensors for p in t.split(STRETCH))
    table, rec, ws = zs.TensorTable(tensors), zs.ClipRecord(), zs.norm_workspace()
    zs.TensorsNorm(table, zs.clip_rule(0.37 * math.sqrt(want)), rec, ws)()
    assert abs(rec.sumsq.item() - want) <= SUM_REL * want, rec.sumsq.item() / want - 1
    assert not ws[:COUNTER_BYTES].any()
    zs.zs_tensors_clip(table, rec)
    assert abs(rec.coef.item() - 0.37) < 1e-6
    for got, old, mask in zip(buffers, before, inside):
        scaled = torch.where(mask, (old.float() * rec.coef).to(old.dtype), old)
        assert torch.equal(got.view(torch.uint8), scaled.view(torch.uint8))


class Shard:
    """Buffers of one rank for one form, from a seed, made on the GPU."""

    def __init__(self, torch, form, n, k, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.form, self.n = form, n
        mv16 = "bf16mv" in form
        moments = torch.bfloat16 if mv16 else torch.float32
        w = torch.empty(n, device="cuda").normal_(0, 0.02, generator=gen)
        m = torch.empty(n, dtype=moments, device="cuda").normal_(0, 1e-2, generator=gen)
        v = torch.empty(n, dtype=moments, device="cuda").uniform_(1e-6, 1e-4, generator=gen)
        if form.startswith("packed"):
            floats = zs.packed_bf16mv_floats(n) if mv16 else zs.packed_floats(n)
            state = torch.zeros(floats, device="cuda")
            pack = zs.zs_pack_state_bf16mv if mv16 else zs.zs_pack_state
            pack(w, m, v, state, n)
            w, m, v = state, None, None
        self.master, self.m, self.v = w, m, v
        self.param = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
        q8 = form.endswith("q8grad")
        self.grads, scales = partials(torch, "int8" if q8 else "bf16", n, k, seed + 1)
        self.more = {"qscales": scales} if q8 else {}
        if form.endswith("q8ag"):
            self.more = dict(param_q8=torch.zeros(n, dtype=torch.int8, device="cuda"),
                             param_q8_scale=torch.zeros(-(-n // 256), device="cuda"))
        if form.endswith("_sr"):
            self.more["seed"] = 77
        cut = n // 3 + 11
        self.table = H.segment_tensor([(0, True), (cut, False), (2 * cut, True)], "cuda")

    def step(self, hp, clip=None):
        return zs.ShardStep(self.master, self.m, self.v, self.param, self.grads, self.n, self.table,
                            hp, variant=self.form, clip=clip, **self.more)

    def outputs(self):
        return [x for x in (self.master, self.m, self.v, self.param, self.more.get("param_q8"),
                            self.more.get("param_q8_scale")) if x is not None]


def clipped_equals_unclipped(torch, form, n, k):
    a, b = (Shard(torch, form, n, k, 5) for _ in range(2))
    rec = zs.ClipRecord()
    zs.GradNorm(a.grads, n, None, rec, 0.25, a.more.get("qscales"))()
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(0.6 * rec.norm.item()), rec)
    coef = np.float32(rec.coef.item())
    assert abs(coef - 0.6) < 1e-6
    a.step(hp_of(0.25), rec)(12)
    b.step(hp_of(float(np.float32(0.25) * coef)))(12)
    for x, y in zip(a.outputs(), b.outputs()):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert bool(a.param.any())


# The clipped step takes the XCD-contiguous order from 4 MB of partials of 8 bytes
# per element on, the unclipped one from 2^26 elements on, then under an occupancy cap.
@pytest.mark.parametrize("form", H.VARIANTS)
@pytest.mark.parametrize("n,k", [(20_000_003, 8), ((1 << 26) + 8 * 5001 + 3, 2)])
def test_large_clipped_steps_equal_the_unclipped(gpu, form, n, k):
    clipped_equals_unclipped(gpu, form, n, k)


@pytest.mark.parametrize("form", ["bf16mv", "packed_bf16mv_sr"])
def test_clipped_steps_past_32_bits_equal_the_unclipped(gpu, form):
    """From 2^32 elements the bf16-moment forms take two sub-windows per wavefront."""
    clipped_equals_unclipped(gpu, form, (1 << 32) + 100_003, 1)
    gpu.cuda.empty_cache()
