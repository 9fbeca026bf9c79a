"""Gradient norm and clipping: cases, their plain form, and the library's calls.

Four operators of a sharded optimizer step:

* ``partials_norm``: the global norm of a shard's reduced gradient (the fold
  of its k partials, bf16 or block-quantized int8, times a scale) and the
  clipping coefficient it gives;
* ``tensors_norm``: the same over a list of tensors of bf16, fp16 and fp32;
* ``tensors_clip``: the coefficient of several ranks' sums of squares, and the
  list scaled by it in place;
* ``clipped_step``: the norm of a shard's partials and the AdamW step on the
  clipped gradient.

``run`` computes them with elementary torch operations, or, where ``own`` is
true, with the calls a user makes of sharded_mixed_precision_shard_amd.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 256      # elements per scale of an int8 partial
EPS = 1e-6       # added to the norm before the quotient
LR, BETA1, BETA2, ADAM_EPS, DECAY = 3e-4, 0.9, 0.95, 1e-8, 0.1
STEP = 101       # the optimizer step t of the bias corrections
SIGMA = 1e-3     # of one partial's elements
RANKS = 8        # sums of squares that a coefficient is formed from
TYPES = {"bf16": (torch.bfloat16,), "fp16": (torch.float16,), "fp32": (torch.float32,),
         "mixed": (torch.bfloat16, torch.float32, torch.float16)}


def listed():
    return [
        # a few thousand parameters on one rank: nothing but latency
        dict(name="norm, small shard", op="partials_norm", form="bf16", n=10007, k=3, ratio=0.5),
        # a 7B model on 8 ranks, one partial of each: heavy-tailed gradients
        dict(name="norm, 7B shard", op="partials_norm", form="bf16", n=805388288, k=8, ratio=0.5),
        # a 175B model on 64 ranks, the partials of a quantized reduce-scatter
        dict(name="norm, 175B shard int8", op="partials_norm", form="int8", n=2718001152, k=2,
             ratio=2.0),
        # replicated norm weights and biases, odd sizes
        dict(name="norm, small tensors", op="tensors_norm", types="fp32", count=41, total=200003,
             layout=1),
        # every gradient of a 0.7B model in bf16
        dict(name="norm, bf16 tensors", op="tensors_norm", types="bf16", count=292,
             total=708297600, layout=2),
        # gradients of three types, as where some layers accumulate in fp32
        dict(name="norm, mixed tensors", op="tensors_norm", types="mixed", count=301,
             total=1600000007, layout=3),
        # the small tensors above, scaled
        dict(name="clip, small tensors", op="tensors_clip", types="fp32", count=41, total=200003,
             layout=1),
        # every gradient of a 0.7B model in bf16, scaled
        dict(name="clip, bf16 tensors", op="tensors_clip", types="bf16", count=292,
             total=708297600, layout=2),
        # a small model's step, four partials
        dict(name="step, small shard", op="clipped_step", form="base", n=1 << 20, k=4, segments=1,
             ratio=0.5),
        # GPT-2-small on 8 ranks: the partials nearly fill the last-level cache
        dict(name="step, GPT-2-small shard", op="clipped_step", form="base", n=15554976, k=8,
             segments=27, ratio=0.5),
        # a 7B model on 8 ranks: the partials are read from memory both times
        dict(name="step, 7B shard", op="clipped_step", form="base", n=805388288, k=8, segments=32,
             ratio=0.5),
        # a 175B model on 64 ranks with bf16 moments
        dict(name="step, 175B shard bf16 moments", op="clipped_step", form="bf16mv", n=2718001152,
             k=2, segments=13, ratio=0.5),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("partials_norm", "tensors_norm", "tensors_clip", "clipped_step"))
    if op == "partials_norm":
        return dict(op=op, form=rng.choice(("bf16", "int8")), n=_between(rng, 100, 4e8),
                    k=rng.randint(1, 16), ratio=rng.choice((0.3, 0.5, 2.0)))
    if op == "clipped_step":
        n = _between(rng, 100, 3e8)
        return dict(op=op, form=rng.choice(("base", "bf16mv")), n=n, k=rng.randint(1, 16),
                    segments=min(n, _between(rng, 1, 2000)), ratio=rng.choice((0.3, 0.5, 2.0)))
    count = _between(rng, 1, 1000)
    return dict(op=op, types=rng.choice(tuple(TYPES)), count=count,
                total=max(count, _between(rng, 1000, 6e8)), layout=rng.randrange(1 << 20))


def _sizes(case):
    """Sizes of a list of tensors: half of them small, the rest sharing what is left."""
    r = np.random.RandomState(case["layout"])
    share = np.where(np.arange(case["count"]) % 2 == 0, 1.0, 1e-3) * r.uniform(0.5, 1.5,
                                                                               case["count"])
    sizes = np.maximum(1, np.floor(share / share.sum() * (case["total"] - case["count"])))
    sizes = sizes.astype(np.int64)
    sizes[0] += case["total"] - int(sizes.sum())
    return [int(x) for x in sizes]


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    device = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    s = dict(case)
    if case["op"] in ("tensors_norm", "tensors_clip"):
        types = TYPES[case["types"]]
        sizes = _sizes(case)
        s["buffers"], s["tensors"] = [], [None] * len(sizes)
        for j, dtype in enumerate(types):
            mine = [i for i in range(len(sizes)) if i % len(types) == j]
            if not mine:
                continue
            flat = torch.empty(sum(sizes[i] for i in mine), dtype=dtype, device=device)
            # fp16 gradients carry a loss scale
            flat.normal_(0.0, 1.0 if dtype == torch.float16 else SIGMA, generator=gen)
            for i, part in zip(mine, flat.split([sizes[i] for i in mine])):
                s["tensors"][i] = part
            s["buffers"].append(flat)
        s["max_norm"] = 0.5 * SIGMA * math.sqrt(case["total"])
        if case["op"] == "tensors_clip":
            # the other ranks' sums of squares, for a coefficient a little under 1
            sums = torch.rand(RANKS, dtype=torch.float64, device=device, generator=gen)
            s["sums"] = (1.02 + 0.04 * sums) * (s["max_norm"] ** 2 / RANKS)
        return s
    n, k = case["n"], case["k"]
    if case["form"] == "int8":
        blocks = -(-n // BLOCK)
        s["codes"] = torch.empty((k, blocks * BLOCK), dtype=torch.int8, device=device)
        s["codes"].random_(-127, 128, generator=gen)
        s["codes"][:, n:] = 0
        s["scales"] = torch.rand((k, blocks), device=device, generator=gen)
        s["scales"].mul_(2e-5).add_(1e-5)
        s["partials"] = [row[:n] for row in s["codes"]]
    else:
        rows = torch.empty((k, -(-n // 8) * 8), dtype=torch.bfloat16, device=device)
        rows.normal_(0.0, SIGMA, generator=gen)
        # one element in a hundred of a heavy tail
        tail = rows[:, int(seed) % 100::100]
        tail.copy_(torch.randn(tail.shape, device=device, generator=gen).mul_(0.1))
        s["grads"] = rows[:, :n]
        s["partials"] = [row[:n] for row in rows]
    s["max_norm"] = case["ratio"] * 0.01 * math.sqrt(k * n)
    if case["op"] == "clipped_step":
        moments = torch.bfloat16 if case["form"] == "bf16mv" else torch.float32
        s["master"] = torch.empty(n, device=device).normal_(0.0, 0.02, generator=gen)
        s["m"] = torch.empty(n, dtype=moments, device=device).normal_(0.0, SIGMA, generator=gen)
        s["v"] = torch.empty(n, dtype=moments, device=device).normal_(0.0, SIGMA, generator=gen)
        s["v"].mul_(s["v"]).add_(SIGMA * SIGMA)
        s["param"] = torch.zeros(n, dtype=torch.bfloat16, device=device)
        cuts = np.random.RandomState(n % (1 << 31)).randint(0, n, case["segments"] - 1)
        starts = [0] + sorted(int(c) for c in cuts)
        flags = [(i + 1) % 2 for i in range(len(starts))]
        s["table"] = torch.tensor([[a, f] for a, f in zip(starts, flags)], dtype=torch.int64,
                                  device=device)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # what a program sets up once beside its buffers
        import sharded_mixed_precision_shard_amd as zs
        device = s["buffers"][0].device if "buffers" in s else s["partials"][0].device
        if zs.zs_init(device.index) != zs.ZS_OK:
            raise RuntimeError("zs_init")
        s["record"] = zs.ClipRecord(device)
        s["rule"] = zs.clip_rule(s["max_norm"], EPS)
        if "buffers" in s:
            s["list"] = zs.TensorTable(s["tensors"])
            if case["op"] == "tensors_norm":
                s["norm"] = zs.TensorsNorm(s["list"], s["rule"], s["record"])
        else:
            scales = list(s["scales"]) if "scales" in s else None
            s["norm"] = zs.GradNorm(s["partials"], case["n"], s["rule"], s["record"],
                                    qscales=scales)
        if case["op"] == "clipped_step":
            s["step"] = zs.ShardStep(s["master"], s["m"], s["v"], s["param"], s["partials"],
                                     case["n"], s["table"],
                                     zs.hparams(LR, BETA1, BETA2, ADAM_EPS, DECAY),
                                     variant=case["form"], clip=s["record"])
    return s


def _coefficient(total, max_norm):
    norm = total.sqrt()
    bound = norm + EPS
    coef = torch.where(bound <= max_norm, torch.ones_like(bound), max_norm / bound)
    return norm.float(), coef.float()


def _reduced(s):
    if "codes" not in s:
        return s["grads"].sum(0, dtype=torch.float32)
    k, blocks = s["scales"].shape
    values = s["codes"].view(k, blocks, BLOCK).float() * s["scales"].unsqueeze(2)
    return values.sum(0).view(-1)[:s["n"]]


def _plain_step(s, g):
    decay = s["table"][:, 1].float() * (LR * DECAY)
    ends = torch.cat((s["table"][1:, 0], s["table"].new_full((1,), s["n"])))
    keep = torch.repeat_interleave(1.0 - decay, ends - s["table"][:, 0], output_size=s["n"])
    m = (s["m"].float() * BETA1).add_(g * (1.0 - BETA1))
    v = (s["v"].float() * BETA2).add_((g * g).mul_(1.0 - BETA2))
    s["m"].copy_(m)
    s["v"].copy_(v)
    update = m.div_(1.0 - BETA1 ** STEP)
    update.div_(v.div_(1.0 - BETA2 ** STEP).sqrt_().add_(ADAM_EPS))
    s["master"].mul_(keep).sub_(update.mul_(LR))
    s["param"].copy_(s["master"])


def run(s):
    op = s["op"]
    if own:
        import sharded_mixed_precision_shard_amd as zs
        stream = torch.cuda.current_stream()
        record = s["record"]
        if op == "tensors_clip":
            zs.zs_clip_combine(s["sums"], s["rule"], record, stream)
            zs.zs_tensors_clip(s["list"], record, stream)
        else:
            s["norm"](stream)
            if op == "clipped_step":
                s["step"](STEP, stream)
        out = {"norm": record.norm, "coef": record.coef}
    else:
        if op == "tensors_clip":
            norm, coef = _coefficient(s["sums"].sum(), s["max_norm"])
            [b.copy_(b.float().mul_(coef)) for b in s["buffers"]]
        elif op == "tensors_norm":
            norm, coef = _coefficient(sum(b.double().square_().sum() for b in s["buffers"]),
                                      s["max_norm"])
        else:
            g = _reduced(s)
            norm, coef = _coefficient(g.double().square_().sum(), s["max_norm"])
            if op == "clipped_step":
                _plain_step(s, g.mul_(coef))
        out = {"norm": norm.view(1), "coef": coef.view(1)}
    if op == "tensors_clip":
        out["tensors"] = s["buffers"]
    if op == "clipped_step":
        out.update(master=s["master"], m=s["m"], v=s["v"], param=s["param"])
    return out


def exact(case, seed):
    """The outputs of one pass in 64 bits, a stretch of elements at a time."""
    s = _inputs(case, seed)
    op, stretch = case["op"], 1 << 26
    if op == "tensors_clip":
        total = math.fsum(s["sums"].tolist())
    elif op == "tensors_norm":
        total = math.fsum(float(torch.dot(x, x)) for t in s["tensors"]
                          for x in (p.double() for p in t.split(stretch)))
    else:
        n = case["n"]

        def gradient(a, b):
            g = torch.zeros(b - a, dtype=torch.float64, device=s["partials"][0].device)
            for j, partial in enumerate(s["partials"]):
                x = partial[a:b].double()
                if "scales" in s:  # stretches begin at a block
                    each = s["scales"][j, a // BLOCK:-(-b // BLOCK)].double()
                    x = x * each.repeat_interleave(BLOCK)[:b - a]
                g += x
            return g

        spans = [(a, min(a + stretch, n)) for a in range(0, n, stretch)]
        total = math.fsum(float(torch.dot(g, g)) for g in (gradient(a, b) for a, b in spans))
    norm = math.sqrt(total)
    coef = min(1.0, s["max_norm"] / (norm + EPS))
    out = {"norm": np.array([norm]), "coef": np.array([coef])}
    if op == "tensors_clip":
        out["tensors"] = [b.double() * coef for b in s["buffers"]]
    if op == "clipped_step":
        for name in ("master", "m", "v"):
            out[name] = torch.empty(n, dtype=torch.float64, device=s["master"].device)
        starts, flags = s["table"][:, 0].contiguous(), s["table"][:, 1]
        for a, b in spans:
            g = gradient(a, b) * coef
            i = torch.arange(a, b, device=g.device)
            on = flags[torch.searchsorted(starts, i, right=True) - 1].bool()
            w = s["master"][a:b].double()
            m = BETA1 * s["m"][a:b].double() + (1 - BETA1) * g
            v = BETA2 * s["v"][a:b].double() + (1 - BETA2) * g ** 2
            step = (m / (1 - BETA1 ** STEP)) / ((v / (1 - BETA2 ** STEP)) ** 0.5 + ADAM_EPS)
            w = torch.where(on, w - LR * DECAY * w, w) - LR * step
            out["master"][a:b], out["m"][a:b], out["v"][a:b] = w, m, v
        out["param"] = out["master"]
    return out


def work(case):
    """Bytes read once and written once, and floating-point operations."""
    if case["op"] in ("tensors_norm", "tensors_clip"):
        types = TYPES[case["types"]]
        size = sum(x * torch.finfo(types[i % len(types)]).bits // 8
                   for i, x in enumerate(_sizes(case)))
        if case["op"] == "tensors_norm":
            return {"bytes": size + 8, "flops": 2 * case["total"]}
        return {"bytes": 2 * size + 8 * RANKS + 8, "flops": case["total"]}
    n, k = case["n"], case["k"]
    read = k * (n + 4 * -(-n // BLOCK)) if case["form"] == "int8" else 2 * k * n
    if case["op"] == "partials_norm":
        adds = (2 * k if case["form"] == "int8" else k) + 1
        return {"bytes": read + 8, "flops": adds * n}
    moments = 4 if case["form"] == "bf16mv" else 8
    state = 4 + moments + 4 + moments + 2
    return {"bytes": read + state * n + 16 * case["segments"] + 8, "flops": (k + 17) * n}
