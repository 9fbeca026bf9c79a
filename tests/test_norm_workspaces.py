"""The one-call norm functions take the caller's workspace and refuse to be
called without one: a workspace of their own would be free again when they
return, while the kernel may still use it.  CPU only: no call gets that far."""
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.test_binding_checks import FakeGpuTensor


class FakeTable:
    device = None
    table = zs.ZsTensorTable(0, 0)


def test_one_call_norms_need_a_workspace():
    n, rec = 1000, FakeGpuTensor(24)
    with pytest.raises(ValueError, match="zs_grad_norm needs a workspace"):
        zs.zs_grad_norm([FakeGpuTensor(2 * n)], 1, n, 1.0, None, rec, None)
    with pytest.raises(ValueError, match="zs_grad_norm_q8grad needs a workspace"):
        zs.zs_grad_norm_q8grad([FakeGpuTensor(n)], [FakeGpuTensor(16)], 1, n, 1.0, None, rec, None)
    with pytest.raises(ValueError, match="zs_tensors_norm needs a workspace"):
        zs.zs_tensors_norm(FakeTable(), None, rec, None)


def test_a_workspace_given_is_taken():
    n, rec, ws = 1000, FakeGpuTensor(24), FakeGpuTensor(zs.ZS_NORM_WORKSPACE_BYTES)
    # null addresses: the library refuses
    for rc in (zs.zs_grad_norm([FakeGpuTensor(2 * n)], 1, n, 1.0, None, rec, ws, check=False),
               zs.zs_tensors_norm(FakeTable(), None, rec, ws, check=False)):
        assert rc == zs.ZS_ERR_INVALID_ARGUMENT
