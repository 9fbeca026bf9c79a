"""Record and workspace made during a graph capture: replays start from their
zeroing, eager calls on them are refused and change nothing, and objects made
before the capture serve both."""
import math

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.test_gpu_norm import check, gpu, on_gpu, partials, reference, widen  # noqa: F401

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-6))


def test_eager_calls_on_a_captures_objects_are_refused(gpu):
    torch, n = gpu, 500_009
    rng = np.random.default_rng(21)
    part = on_gpu(torch, partials(rng, n, 1)[0])
    x = torch.randn(5000, device="cuda")
    table, before = zs.TensorTable([x]), x.clone()
    early = zs.ClipRecord()
    norm_early = zs.GradNorm([part], n, zs.clip_rule(1.0), early)
    norm_early()                           # the kernel is loaded before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rec, ws = zs.ClipRecord(), zs.norm_workspace()
        norm = zs.GradNorm([part], n, zs.clip_rule(1.0), rec, workspace=ws)
        norm(torch.cuda.current_stream())
        norm_early(torch.cuda.current_stream())

    def refused():
        other = zs.ClipRecord()
        for call in (norm, zs.GradNorm([part], n, None, other, workspace=ws),
                     zs.TensorsNorm(table, None, other, ws),
                     lambda: zs.zs_clip_combine(early.sumsq, None, rec),
                     lambda: zs.zs_tensors_clip(table, rec)):
            with pytest.raises(ValueError, match="made during a graph capture"):
                call()
        torch.cuda.synchronize()
        assert other.apply.item() == 0 and torch.equal(x, before)

    refused()                              # before the first replay
    for _ in range(4):
        bits = partials(rng, n, 1)[0]
        part[:n] = torch.from_numpy(bits.view(np.int16)).cuda()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = reference(widen(bits), 1.0, EPS)
        check(rec, *want)
        check(early, *want)
        early.buffer.zero_()
        norm_early()                       # made before the capture: eager, too
        check(early, *want)
        assert torch.isfinite(torch.randn(4096, device="cuda").square().sum())
        torch.cuda.synchronize()
    refused()                              # and after
    assert math.isfinite(rec.norm.item())
