"""The clipping recipes of README.md, run as they are printed on a stream that is
not torch's current one, as one of three ranks (the all-reduce, a stand-in, finds
the same sum on each), against the unclipped step with the coefficient in its
grad_scale.

Tolerance.  The total and its norm as in the norm's own tests; the product with
the three ranks is one rounding of binary64 more, far below 2^-34."""
import math
import os
import re

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.conftest import ROOT
from tests.test_gpu_clipped_step import Shard, hp_of, same
from tests.test_gpu_norm import REL, fold, gpu, reference, rule_of  # noqa: F401

pytestmark = pytest.mark.gpu

N, K, T, RANKS, SCALE = 70_001, 3, 12, 3, 0.25


def recipes():
    text = open(os.path.join(ROOT, "README.md")).read()
    return [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "zs." in b]


@pytest.fixture
def job(gpu, monkeypatch):
    """What a program has in hand before the recipes, as their names."""
    torch, stream = gpu, gpu.cuda.Stream()
    s = Shard(torch, "base", N, K, 9)
    s.tensors = [torch.randn(777, device="cuda"), torch.randn(64, 9, device="cuda").half()]
    stream.wait_stream(torch.cuda.current_stream())

    def all_reduce(x):
        # a collective orders itself with the current stream
        assert torch.cuda.current_stream() == stream
        x.mul_(RANKS)

    monkeypatch.setattr(torch.distributed, "all_reduce", all_reduce)
    names = dict(zs=zs, torch=torch, device="cuda", stream=stream, partials=s.grads, n=N, k=K, t=T,
                 master=s.master, m=s.dm, v=s.dv, param=s.param, segments=s.table,
                 hparams=hp_of(SCALE), grad_scale=SCALE, tensors=s.tensors, lr=1e-3, beta1=0.9,
                 beta2=0.95, eps=1e-8, decay=0.1, host_master=s.w.copy(), host_m=s.m.copy(),
                 host_v=s.v.copy(), host_param=np.zeros(N, np.uint16), host_partials=s.bits,
                 host_segments=s.segs)
    return torch, s, names


def test_one_total_over_the_ranks(job):
    torch, s, names = job
    exec(recipes()[0], names)
    torch.cuda.synchronize()
    total = RANKS * reference(fold(s.values, SCALE))[0]
    _, coef = rule_of(total, 1.0, float(np.float32(1e-6)))
    got = names["record"].coef.item()
    assert coef < 1 and abs(got - coef) <= REL * coef
    other = Shard(torch, "base", N, K, 9)
    other.step(hp_of(float(np.float32(SCALE) * np.float32(got))))(T)
    assert same(torch, s.outputs(), other.outputs())


def test_tensors_outside_the_shard_count_once(job):
    torch, s, names = job
    before = [x.clone() for x in s.tensors]
    exec(recipes()[0].split("with torch")[0], names)
    exec(recipes()[1], names)
    torch.cuda.synchronize()
    total = RANKS * reference(fold(s.values, SCALE))[0] + \
        sum(reference(x.double().cpu().numpy())[0] for x in before)
    norm, coef = rule_of(total, 1.0, float(np.float32(1e-6)))
    record = names["record"]
    assert abs(record.norm.item() - norm) <= REL * norm
    assert coef < 1 and abs(record.coef.item() - coef) <= REL * coef
    for x, b in zip(s.tensors, before):
        assert torch.equal(x, (b.float() * record.coef).to(b.dtype))
    other = Shard(torch, "base", N, K, 9)
    other.step(hp_of(float(np.float32(SCALE) * np.float32(record.coef.item()))))(T)
    assert same(torch, s.outputs(), other.outputs())


def test_host_step_and_its_skip(job):
    torch, s, names = job
    hosts = [names["host_" + x] for x in ("master", "m", "v", "param")]
    start = [h.copy() for h in hosts]
    exec(recipes()[0], names)
    exec(recipes()[2], names)
    for dev, host in zip((s.master, s.dm, s.dv, s.param), hosts):
        assert np.array_equal(dev.cpu().numpy().view(np.uint8), host.view(np.uint8))
    # an infinity: nothing steps, on the device or the host
    for h, a in zip(hosts, start):
        h[...] = a
    device = [x.clone() for x in s.outputs()]
    s.grads[1][N - 1] = 0x7f80
    s.bits[1][N - 1] = 0x7f80
    torch.cuda.synchronize()
    exec(recipes()[0], names)
    exec(recipes()[2], names)
    torch.cuda.synchronize()
    assert names["record"].norm.item() == math.inf and names["record"].apply.item() == 0
    assert same(torch, s.outputs(), device)
    for h, a in zip(hosts, start):
        assert np.array_equal(h.view(np.uint8), a.view(np.uint8))
