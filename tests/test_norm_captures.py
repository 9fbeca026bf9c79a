"""A record or workspace made during a graph capture holds anything until that
graph's first replay: eager calls on it are refused.  CPU only, with stand-ins."""
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.test_binding_checks import FakeGpuTensor
from tests.test_norm_workspaces import FakeTable

N = 1000


def marked(nbytes):
    x = FakeGpuTensor(nbytes)
    x.made_in_capture = True
    return x


def calls(clip, workspace):
    """Every call that takes a record or a workspace, by name (null addresses:
    the library refuses whatever reaches it)."""
    g, f = [FakeGpuTensor(2 * N)], [FakeGpuTensor(4 * N) for _ in range(3)] + [FakeGpuTensor(2 * N)]
    st = zs.seg_table(FakeGpuTensor(16), 1)
    return {
        "zs_grad_norm": lambda: zs.GradNorm(g, N, None, clip, workspace=workspace)(check=False),
        "zs_grad_norm ": lambda: zs.zs_grad_norm(g, 1, N, 1.0, None, clip, workspace, check=False),
        "zs_tensors_norm": lambda: zs.TensorsNorm(FakeTable(), None, clip, workspace)(check=False),
        "zs_clip_combine": lambda: zs.zs_clip_combine(0, None, clip, count=1, check=False),
        "zs_tensors_clip": lambda: zs.zs_tensors_clip(FakeTable(), clip, check=False),
        "ShardStep": lambda: zs.ShardStep(*f, g, N, st, zs.hparams(), clip=clip)(1, check=False),
    }


def test_eager_calls_on_what_a_capture_made_are_refused(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ws = FakeGpuTensor(zs.ZS_NORM_WORKSPACE_BYTES)
    for name, call in calls(marked(24), ws).items():
        with pytest.raises(ValueError, match="made during a graph capture"):
            call()
    # the workspace alone
    made = calls(FakeGpuTensor(24), marked(zs.ZS_NORM_WORKSPACE_BYTES))
    for name in ("zs_grad_norm", "zs_grad_norm ", "zs_tensors_norm"):
        with pytest.raises(ValueError, match="made during a graph capture"):
            made[name]()
    # neither: on to the library
    for name, call in calls(FakeGpuTensor(24), ws).items():
        assert call() in (zs.ZS_ERR_INVALID_ARGUMENT, zs.ZS_ERR_NOT_INITIALIZED), name


def test_calls_inside_a_capture_are_taken(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    for name, call in calls(marked(24), marked(zs.ZS_NORM_WORKSPACE_BYTES)).items():
        assert call() in (zs.ZS_ERR_INVALID_ARGUMENT, zs.ZS_ERR_NOT_INITIALIZED), name
