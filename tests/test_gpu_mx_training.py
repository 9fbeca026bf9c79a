"""A training step on the microscaled formats as a program makes it: the 4-bit copy of
the parameters, two linear layers on its blocks, their inputs kept in 8 bits, the
weights' gradients made from those as the partial that norm and clipped step take.

Every stage is held against a plain implementation in 64 bits on the inputs that the stage
had.  Tolerances: codes, scales and the step are exact; an fp32 sum of C exact products is
within C 2^-23 sum|p|, a bf16 output of it half a step, 2^-8, more."""
import os
import re

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests import _mx_reference as ref
from tests.conftest import ROOT
from tests.test_gpu_norm import gpu  # noqa: F401

pytestmark = pytest.mark.gpu

M, D0, D1, D2, TAIL = 33, 64, 96, 40, 7
SIZE = D1 * D0 + D2 * D1 + TAIL
T = 5


class Net:
    """Weights [D1, D0] and [D2, D1] in one flat shard, a few more elements behind them."""

    def __init__(self, torch, seed, stream=None):
        self.torch = torch
        gen = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0, dtype=torch.float32):
            return (torch.randn(*shape, generator=gen) * scale).to(dtype).cuda()

        self.master = normal(SIZE, scale=0.1)
        self.m, self.v = normal(SIZE, scale=1e-3), normal(SIZE, scale=1e-3).square()
        self.param = self.master.to(torch.bfloat16)
        self.x = normal(M, D0, dtype=torch.bfloat16)
        self.target = normal(M, D2)
        self.partial = torch.zeros(SIZE, dtype=torch.bfloat16, device="cuda")
        self.dw1 = self.partial[:D1 * D0].view(D1, D0)
        self.dw2 = self.partial[D1 * D0:D1 * D0 + D2 * D1].view(D2, D1)
        self.y1 = torch.empty(M, D1, dtype=torch.bfloat16, device="cuda")
        self.y2 = torch.empty(M, D2, device="cuda")
        self.dy1 = torch.empty(M, D1, dtype=torch.bfloat16, device="cuda")
        self.copy = zs.Mx.empty(1, SIZE, "fp4")
        self.w1 = self.copy.part(0, D1, D0)
        self.w2 = self.copy.part(D1 * D0, D2, D1)
        self.kept0, self.kept1 = zs.Mx.empty(M, D0, "fp8"), zs.Mx.empty(M, D1, "fp8")
        self.space = zs.mx_workspace()
        self.record = zs.ClipRecord()
        self.norm = zs.GradNorm([self.partial], SIZE, zs.clip_rule(0.25), self.record)
        self.table = torch.tensor([[0, 1], [D1 * D0, 0]], dtype=torch.int64, device="cuda")
        self.step = zs.ShardStep(self.master, self.m, self.v, self.param, [self.partial], SIZE,
                                 self.table, zs.hparams(), clip=self.record)

    def state(self):
        return [t.clone() for t in (self.master, self.m, self.v, self.param)]

    def run(self):
        torch, s = self.torch, self.torch.cuda.current_stream()
        zs.zs_mx_quantize(self.param, self.copy, s)
        zs.zs_mx_quantize(self.x, self.kept0, s)
        zs.zs_mx_linear(self.x, self.w1, self.y1, s, self.space)
        zs.zs_mx_quantize(self.y1, self.kept1, s)
        zs.zs_mx_product(self.kept1, self.w2, self.y2, s, self.space)
        self.dy2 = ((self.y2 - self.target) * (1.0 / M)).to(torch.bfloat16)
        zs.zs_mx_linear_wgrad(self.dy2, self.kept1, self.dw2, False, s, self.space)
        zs.zs_mx_linear_dgrad(self.dy2, self.w2, self.dy1, s, self.space)
        zs.zs_mx_linear_wgrad(self.dy1, self.kept0, self.dw1, False, s, self.space)
        self.norm(s)
        self.step(T, s)


def double(x):
    return x.double().cpu().numpy()


def near(got, a, b):
    """got = a @ b within what its sums and its type may be off by."""
    want, sizes = a @ b, np.abs(a) @ np.abs(b)
    room = a.shape[1] * 2.0 ** -23 * sizes
    if got.element_size() == 2:
        room = room + 2.0 ** -8 * (np.abs(want) + room)
    assert (np.abs(double(got) - want) <= room).all()


def values(mx):
    return ref.decode(mx.codes.cpu().numpy(), mx.scales.cpu().numpy(), mx.format, mx.cols)


def held_equal(mx, x, fmt):
    codes, scales = ref.encode(double(x).reshape(mx.rows, mx.cols), fmt)
    assert np.array_equal(mx.codes.cpu().numpy().reshape(codes.shape), codes)
    assert np.array_equal(mx.scales.cpu().numpy().reshape(scales.shape), scales)


def test_three_steps(gpu):
    torch = gpu
    net = Net(torch, 1)
    for _ in range(3):
        before = net.state()
        net.run()
        torch.cuda.synchronize()
        held_equal(net.copy, before[3], "fp4")
        held_equal(net.kept0, net.x, "fp8")
        held_equal(net.kept1, net.y1, "fp8")
        w1, w2, x0, x1 = (values(h) for h in (net.w1, net.w2, net.kept0, net.kept1))
        flat = values(net.copy)[0]
        assert np.array_equal(w1.reshape(-1), flat[:D1 * D0])
        assert np.array_equal(w2.reshape(-1), flat[D1 * D0:SIZE - TAIL])
        near(net.y1, double(net.x), w1.T)
        near(net.y2, x1, w2.T)
        near(net.dw2, double(net.dy2).T, x1)
        near(net.dy1, double(net.dy2), w2)
        near(net.dw1, double(net.dy1).T, x0)
        assert not net.partial[SIZE - TAIL:].any()
        # the clipped step: the step with the record's coefficient in its grad_scale
        coef = net.record.coef.item()
        assert 0 < coef < 1
        zs.zs_shard_step(*before, [net.partial], 1, SIZE, zs.seg_table(net.table),
                         zs.hparams(grad_scale=coef), T, torch.cuda.current_stream())
        for got, want in zip(net.state(), before):
            assert torch.equal(got, want)


def test_captured_step_equals_eager(gpu):
    """The whole step as one graph, replayed on other inputs between eager work."""
    torch = gpu
    net = Net(torch, 2)
    start = net.state()
    net.run()                                 # kernels are loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        net.run()
    for seed in range(4):
        net.x.copy_(torch.randn(M, D0, generator=torch.Generator().manual_seed(seed)))

        def reset():
            for to, of in zip((net.master, net.m, net.v, net.param), start):
                to.copy_(of)
            net.partial.zero_()

        reset()
        net.run()
        torch.cuda.synchronize()
        want, grads = net.state(), net.partial.clone()
        reset()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(net.partial, grads)
        for got, ok in zip(net.state(), want):
            assert torch.equal(got, ok)
        torch.randn(4096, device="cuda").square().sum().item()


def test_two_streams_with_a_workspace_each(gpu):
    """Products that split their sums, side by side: each as it is alone."""
    torch = gpu
    sides, work = [torch.cuda.Stream(), torch.cuda.Stream()], []
    for i in range(2):
        gen = torch.Generator().manual_seed(i)
        x = torch.randn(100 + i, 8192, generator=gen).to(torch.bfloat16).cuda()
        w = zs.Mx.empty(200, 8192, "fp4")
        zs.zs_mx_quantize(torch.randn(200, 8192, generator=gen).cuda(), w)
        space = zs.mx_workspace()
        alone = torch.empty(100 + i, 200, device="cuda")
        torch.cuda.synchronize()
        zs.zs_mx_linear(x, w, alone, torch.cuda.current_stream(), space)
        work.append((x, w, space, alone, [torch.empty_like(alone) for _ in range(20)]))
    torch.cuda.synchronize()
    for n in range(20):
        for side, (x, w, space, _, outs) in zip(sides, work):
            zs.zs_mx_linear(x, w, outs[n], side, space)
    torch.cuda.synchronize()
    for _, _, space, alone, outs in work:
        assert all(torch.equal(o, alone) for o in outs)
        assert not space[:65536].any()


def test_buffers_of_a_device_that_is_not_current_are_refused(gpu, monkeypatch):
    torch = gpu
    x = torch.zeros(4, 32, device="cuda")
    held = zs.Mx.empty(4, 32, "fp4")
    monkeypatch.setattr(zs, "_current_device", lambda: 7)
    with pytest.raises(ValueError, match="current device"):
        zs.zs_mx_quantize(x, held)


def test_the_readme_recipe(gpu, monkeypatch):
    """The recipe of README.md as it is printed, on one of two ranks whose shards are alike (the
    all-gather, a stand-in, finds the same blocks on both), on a stream of its own."""
    torch = gpu
    text = open(os.path.join(ROOT, "README.md")).read()
    recipe, = [b for b in re.findall(r"```python\n(.*?)```", text, re.S) if "zs_mx_linear" in b]
    stream = torch.cuda.Stream()

    def all_gather_into_tensor(out, mine):
        assert torch.cuda.current_stream() == stream
        out.copy_(mine.expand_as(out))

    monkeypatch.setattr(torch.distributed, "all_gather_into_tensor", all_gather_into_tensor)
    gen = torch.Generator().manual_seed(3)
    n, ranks, tokens, inputs, outputs, start = 6400, 2, 50, 96, 70, 3200
    param = torch.randn(n, generator=gen).to(torch.bfloat16).cuda()
    x = torch.randn(tokens, inputs, generator=gen).to(torch.bfloat16).cuda()
    dy = torch.randn(tokens, outputs, generator=gen).to(torch.bfloat16).cuda()
    partial = torch.zeros(n * ranks, dtype=torch.bfloat16, device="cuda")
    names = dict(zs=zs, torch=torch, device="cuda", stream=stream, n=n, ranks=ranks, param=param,
                 tokens=tokens, inputs=inputs, outputs=outputs, start=start, x=x, dy=dy,
                 y=torch.empty(tokens, outputs, dtype=torch.bfloat16, device="cuda"),
                 dx=torch.empty(tokens, inputs, dtype=torch.bfloat16, device="cuda"),
                 dw=partial[start:start + outputs * inputs].view(outputs, inputs))
    torch.cuda.synchronize()
    exec(recipe, names)
    torch.cuda.synchronize()
    held = ref.decode(*ref.encode(double(param)[None], "fp4"), "fp4", n)[0]
    w = np.tile(held, ranks)[start:start + outputs * inputs].reshape(outputs, inputs)
    kept = ref.decode(*ref.encode(double(x), "fp8"), "fp8", inputs)
    near(names["y"], double(x), w.T)
    near(names["dx"], double(dy), w)
    near(names["dw"], double(dy).T, kept)
    assert not partial[:start].any() and not partial[start + outputs * inputs:].any()
