"""The shard step on the clipped gradient, for every entry point's form: bit for
bit the unclipped step with grad_scale * coef, the oracle's step on the same,
skipped whole where the record says so, captured together with its norm; and
norm, combination and step run together as the ranks of one job would, against
the same training steps in 64 bits."""
import math

import numpy as np
import pytest

import oracle
import sharded_mixed_precision_shard_amd as zs
from tests import _gpu_harness as H
from tests.test_gpu_norm import bf16_bits, fold, gpu, reference, widen  # noqa: F401

pytestmark = pytest.mark.gpu

F32 = np.float32
SEED = 0xC0FFEE


class Shard:
    """Buffers of one rank for one form, from a seed, and its step's arguments."""

    def __init__(self, torch, form, n, k, seed, sigma=1e-2):
        rng = np.random.default_rng(seed)
        self.form, self.n, self.k = form, n, k
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.w = rng.normal(0, 0.02, n).astype(F32)
        self.m = rng.normal(0, sigma, n).astype(F32)
        self.v = (rng.normal(0, sigma, n) ** 2 + 1e-8).astype(F32)
        mv16 = "bf16mv" in form
        if mv16:
            self.m, self.v = bf16_bits(self.m), bf16_bits(self.v)
        pack = H.pack16_host if mv16 else H.pack_host
        half = (lambda a: a.view(np.int16)) if mv16 else (lambda a: a)
        packed = form.startswith("packed")
        self.master = dev(pack(self.w, self.m, self.v) if packed else self.w)
        self.dm = None if packed else dev(half(self.m))
        self.dv = None if packed else dev(half(self.v))
        self.param = torch.zeros(n, dtype=torch.int16, device="cuda")
        self.more = {}
        nb = -(-n // zs.ZS_Q8_BLOCK)
        if form.endswith("q8ag"):
            self.more = dict(param_q8=torch.zeros(n, dtype=torch.int8, device="cuda"),
                             param_q8_scale=torch.zeros(nb, dtype=torch.float32, device="cuda"))
        if form.endswith("q8grad"):
            self.codes = [rng.integers(-127, 128, n).astype(np.int8) for _ in range(k)]
            self.scales = [rng.uniform(1e-5, 1e-4, nb).astype(F32) for _ in range(k)]
            self.more["qscales"] = [dev(s) for s in self.scales]
            self.grads = [dev(c) for c in self.codes]
            self.values = [c.astype(F32) * np.repeat(s, 256)[:n]
                           for c, s in zip(self.codes, self.scales)]
        else:
            self.bits = [bf16_bits(rng.normal(0, sigma, n)) for _ in range(k)]
            self.grads = [dev(b.view(np.int16)) for b in self.bits]
            self.values = [widen(b) for b in self.bits]
        if form.endswith("_sr"):
            self.more["seed"] = SEED
        self.segs, a = [], 0
        while a < n:
            self.segs.append((a, bool(rng.random() < 0.5)))
            a += int(rng.integers(1, max(2, n // 7)))
        self.table = H.segment_tensor(self.segs, "cuda")

    def step(self, hp, clip=None):
        return zs.ShardStep(self.master, self.dm, self.dv, self.param, self.grads, self.n,
                            self.table, hp, variant=self.form, clip=clip, **self.more)

    def norm(self, rule, clip, grad_scale=1.0):
        return zs.GradNorm(self.grads, self.n, rule, clip, grad_scale, self.more.get("qscales"))

    def outputs(self):
        return [x for x in (self.master, self.dm, self.dv, self.param, self.more.get("param_q8"),
                            self.more.get("param_q8_scale")) if x is not None]


def same(torch, a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def hp_of(grad_scale):
    return zs.hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, grad_scale)


@pytest.mark.parametrize("form", H.VARIANTS)
@pytest.mark.parametrize("n,k", [(1, 1), (255, 2), (257, 3), (1000, 16), (100003, 4), (600_011, 8)])
def test_every_form_equals_the_unclipped_step_on_the_scaled_gradient(gpu, form, n, k):
    torch = gpu
    for t in (3, 200, 10000):        # all three kernels of the bias corrections
        a, b = (Shard(torch, form, n, k, 7 * n + k) for _ in range(2))
        s, norm, _ = reference(fold(a.values, 0.25))
        for max_norm in (0.3 * norm, 3 * norm):
            rec = zs.ClipRecord()
            a.norm(zs.clip_rule(max_norm), rec, 0.25)()
            a.step(hp_of(0.25), rec)(t)
            coef = F32(rec.coef.item())
            assert (coef < 1) == (max_norm < norm)
            b.step(hp_of(float(F32(0.25) * coef)))(t)
            assert same(torch, a.outputs(), b.outputs())


@pytest.mark.parametrize("form", ["base", "bf16mv", "q8grad"])
def test_equal_to_the_oracle(gpu, form):
    torch, n, k, t = gpu, 70001, 5, 12
    s = Shard(torch, form, n, k, 5)
    rec = zs.ClipRecord()
    s.norm(zs.clip_rule(0.5), rec)()
    s.step(hp_of(1.0), rec)(t)
    norm = reference(fold(s.values, 1.0))[1]
    assert abs(rec.coef.item() - 0.5 / (norm + float(F32(1e-6)))) <= 2.0 ** -23 * rec.coef.item()
    hp = oracle.hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, rec.coef.item())
    p = np.zeros(n, np.uint16)
    if form == "q8grad":
        rc = oracle.shard_step_q8grad(s.w, s.m, s.v, p, s.codes, s.scales, s.segs, hp, t)
    elif form == "bf16mv":
        rc = oracle.shard_step_bf16mv(s.w, s.m, s.v, p, s.bits, s.segs, hp, t)
    else:
        rc = oracle.shard_step(s.w, s.m, s.v, p, s.bits, s.segs, hp, t)
    assert rc == 0
    for got, want in zip(s.outputs(), (s.w, s.m, s.v, p)):
        assert np.array_equal(got.cpu().numpy().view(np.uint8), want.view(np.uint8))


@pytest.mark.parametrize("form", H.VARIANTS)
def test_a_skipped_step_changes_nothing(gpu, form):
    torch, n = gpu, 5000
    s = Shard(torch, form, n, 2, 3)
    before = [x.clone() for x in s.outputs()]
    rec = zs.ClipRecord()
    s.step(hp_of(1.0), rec)(9)                       # a record no norm call has written
    torch.cuda.synchronize()
    assert same(torch, s.outputs(), before)
    if "q8grad" in form:
        s.more["qscales"][1][7] = math.inf
    else:
        s.grads[1][n - 1] = 0x7f80                   # an infinity in the last element
    s.norm(zs.clip_rule(1.0, skip_nonfinite=True), rec)()
    s.step(hp_of(1.0), rec)(9)
    torch.cuda.synchronize()
    assert rec.apply.item() == 0 and not math.isfinite(rec.norm.item())
    assert same(torch, s.outputs(), before)
    # without the rule's flag the step runs, and what was infinite ends as NaN
    s.norm(zs.clip_rule(1.0), rec)()
    s.step(hp_of(1.0), rec)(9)
    torch.cuda.synchronize()
    assert rec.apply.item() == 1 and not same(torch, s.outputs(), before)


def test_norm_and_step_in_one_graph(gpu):
    """Every replay clips by the norm of the gradient it finds."""
    torch, n, k = gpu, 60_007, 3
    a, b = (Shard(torch, "base", n, k, 17) for _ in range(2))
    rec, rec_b, rule = zs.ClipRecord(), zs.ClipRecord(), zs.clip_rule(0.7)
    norm, step = a.norm(rule, rec), a.step(hp_of(1.0), rec)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm(torch.cuda.current_stream())
        step(50, torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert same(torch, a.outputs(), b.outputs())     # the capture ran nothing
    norm_b, step_b = b.norm(rule, rec_b), b.step(hp_of(1.0), rec_b)
    rng = np.random.default_rng(2)
    for rep in range(4):
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.from_numpy(bf16_bits(rng.normal(0, 10.0 ** -rep, n)).view(np.int16)))
            y.copy_(x)
        torch.cuda.synchronize()
        graph.replay()
        norm_b()
        step_b(50)
        torch.cuda.synchronize()
        assert torch.isfinite(torch.randn(4096, device="cuda").square().sum())
        torch.cuda.synchronize()
        assert torch.equal(rec.buffer, rec_b.buffer) and same(torch, a.outputs(), b.outputs())
        # the norm is near 10^-rep sqrt(3 n) = 424 10^-rep: above the limit but in the last replay
        assert (rec.coef.item() < 1.0) == (rep < 3)


def test_ranks_of_one_job(gpu):
    """Four ranks' shards and a list of replicated tensors, six steps: each
    rank's sum of squares, their total with the replicated tensors', one
    coefficient, every rank's step; against the same in 64 bits.

    Tolerance.  The partials are small multiples of 2^-12, so their fold is
    exact; g is one rounding (2^-24 relative) of coef * fold, and coef is within
    2^-24 + 2^-34 of its value.  One moment update is two products, one sum and
    g's own error: at most 5 roundings of terms whose sizes add up to A = beta1 A
    + (1 - beta1) |g|, so after t steps |dm| <= 5 t 2^-24 A, and v, a sum of
    positive terms with g twice, is within 8 t 2^-24 relative.  u = (m / bc1) /
    (sqrt(v / bc2) + eps) adds 5 roundings and half of v's error.  w then adds the
    error of lr u, and 3 roundings of values no larger than |w| + lr |u|."""
    torch = gpu
    n, k, ranks, steps, e = 5003, 3, 4, 6, 2.0 ** -24
    rng = np.random.default_rng(44)
    shards = [Shard(torch, "base", n, k, r) for r in range(ranks)]
    extra = [torch.zeros(777, device="cuda"), torch.zeros(64, 9, device="cuda")]
    table = zs.TensorTable(extra)
    rule = zs.clip_rule(0.9, 1e-6)
    recs, rec_x = [zs.ClipRecord() for _ in range(ranks)], zs.ClipRecord()
    norms = [s.norm(None, r) for s, r in zip(shards, recs)]
    norm_x = zs.TensorsNorm(table, None, rec_x)
    lr, b1, b2, eps, wd = (float(F32(x)) for x in (1e-3, 0.9, 0.95, 1e-8, 0.1))
    ref = []
    for s in shards:
        s.dm.zero_()
        s.dv.zero_()
        z = np.zeros(n)
        ref.append(dict(w=s.w.astype(np.float64), m=z, v=z, a=z, tol=z))
    stepper = [s.step(zs.hparams(lr, b1, b2, eps, wd), r) for s, r in zip(shards, recs)]
    clipped = 0
    for t in range(1, steps + 1):
        size = 60 if t % 2 else 1                        # every other step is under the limit
        total, folds = 0.0, []
        for s in shards:
            ints = [rng.integers(-size, size + 1, n) for _ in range(k)]
            for g, x in zip(s.grads, ints):
                g.copy_(torch.from_numpy(bf16_bits(x * 2.0 ** -12).view(np.int16)))
            folds.append(sum(ints) * 2.0 ** -12)
            total += float(np.sum(folds[-1] ** 2))
        for x in extra:
            x.copy_(torch.from_numpy(rng.integers(-size, size + 1, tuple(x.shape)) * 2.0 ** -12))
        host = [x.cpu().double().numpy() for x in extra]
        total += float(sum(np.sum(x ** 2) for x in host))
        # the device's run
        for f in (*norms, norm_x):
            f()
        sums = torch.cat([r.sumsq for r in (*recs, rec_x)])
        for r in (*recs, rec_x):
            zs.zs_clip_combine(sums, rule, r)
        for f in stepper:
            f(t)
        zs.zs_tensors_clip(table, rec_x)
        # the same in 64 bits
        d = math.sqrt(total) + float(rule.eps)
        coef = 1.0 if d <= float(rule.max_norm) else float(rule.max_norm) / d
        clipped += coef < 1
        for r in recs:
            assert abs(r.coef.item() - coef) <= (e + 2.0 ** -34) * coef
        for s, q, f in zip(shards, ref, folds):
            g = f * coef
            on = np.zeros(n, bool)
            for i, (a, flag) in enumerate(s.segs):
                on[a:] = flag
            q["m"], q["v"] = b1 * q["m"] + (1 - b1) * g, b2 * q["v"] + (1 - b2) * g * g
            q["a"] = b1 * q["a"] + (1 - b1) * np.abs(g)
            root = np.sqrt(q["v"] / (1 - b2 ** t)) + eps
            u = q["m"] / (1 - b1 ** t) / root
            du = e * (5 * t * q["a"] / (1 - b1 ** t) / root + (4 * t + 8) * np.abs(u))
            q["w"] = np.where(on, q["w"] * (1 - lr * wd), q["w"]) - lr * u
            q["tol"] = q["tol"] + lr * du + 3 * e * (np.abs(q["w"]) + lr * np.abs(u))
        for x, h in zip(extra, host):
            err = np.abs(x.cpu().double().numpy() - h * coef)
            assert (err <= 3 * e * np.abs(h * coef)).all()
    assert clipped == steps // 2
    for s, q in zip(shards, ref):
        w = s.master.cpu().numpy().astype(np.float64)
        assert (np.abs(w - q["w"]) <= 1.01 * q["tol"]).all()
        m = s.dm.cpu().numpy().astype(np.float64)
        assert (np.abs(m - q["m"]) <= 5.05 * steps * e * q["a"]).all()
        v = s.dv.cpu().numpy().astype(np.float64)
        assert (np.abs(v - q["v"]) <= 8.08 * steps * e * q["v"]).all()
        p = widen(s.param.cpu().numpy().view(np.uint16)).astype(np.float64)
        assert (np.abs(p - q["w"]) <= 2.0 ** -8 * np.abs(q["w"]) + 1.02 * q["tol"]).all()


def test_refusals(gpu):
    torch, n = gpu, 1000
    s = Shard(torch, "base", n, 2, 1)
    before = [x.clone() for x in s.outputs()]
    lib, hp, rec = zs.load_library(), hp_of(1.0), zs.ClipRecord()
    b = s.step(hp, rec)._buffers
    st = zs.seg_table(s.table)
    import ctypes

    def call(variant=0, buffers=b, clip=rec.buffer.data_ptr(), k=2):
        return lib.zs_shard_step_clipped(variant, ctypes.byref(buffers) if buffers else None, k, n,
                                         ctypes.byref(st), ctypes.byref(hp), 1, 0, clip, None)
    assert call() == zs.ZS_OK                       # the record is new: nothing happens
    assert call(variant=3) == zs.ZS_ERR_INVALID_ARGUMENT
    assert call(variant=8 + 4) == zs.ZS_ERR_INVALID_ARGUMENT
    assert call(variant=1) == zs.ZS_ERR_INVALID_ARGUMENT      # no int8 copy given
    assert call(variant=2) == zs.ZS_ERR_INVALID_ARGUMENT      # no int8 partials given
    assert call(buffers=None) == zs.ZS_ERR_INVALID_ARGUMENT
    assert call(clip=None) == zs.ZS_ERR_INVALID_ARGUMENT
    assert call(k=0) == zs.ZS_ERR_INVALID_ARGUMENT
    assert call(clip=rec.buffer.data_ptr() + 4) == zs.ZS_ERR_MISALIGNED
    assert call(clip=s.master.data_ptr() + 80) == zs.ZS_ERR_ALIASING
    assert call(clip=s.param.data_ptr() + 2 * n - 8) == zs.ZS_ERR_ALIASING
    with pytest.raises(ValueError, match="needs a record"):
        zs.zs_shard_step_clipped("base", s.master, s.dm, s.dv, s.param, s.grads, n, st, hp, 1, None)
    with pytest.raises(ValueError, match="no launch cfg"):
        zs.ShardStep(s.master, s.dm, s.dv, s.param, s.grads, n, st, hp, cfg=dict(chunk_tiles=2),
                     clip=rec)
    torch.cuda.synchronize()
    assert same(torch, s.outputs(), before)
    # the one-call form
    rec.sumsq.fill_(4.0)
    zs.zs_clip_combine(rec.sumsq, zs.clip_rule(1.0, 0.0), rec)
    zs.zs_shard_step_clipped("base", s.master, s.dm, s.dv, s.param, s.grads, n, st, hp, 1, rec)
    other = Shard(torch, "base", n, 2, 1)
    other.step(hp_of(0.5))(1)
    assert same(torch, s.outputs(), other.outputs())
