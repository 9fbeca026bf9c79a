"""What a record holds where a norm is not finite, as the header states it, for
each of the calls that write one, and what the scaling then does.  Tolerances as
in the norm's own tests: coef is one rounding of its 64-bit value, which may lie
under binary32's normal range (half a step there: 2^-150)."""
import math

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.test_gpu_norm import (F32_MAX, bf16_bits, check, close, gpu, on_gpu,  # noqa: F401
                                 reference, widen)

pytestmark = pytest.mark.gpu

BIG = [2.0 ** 127] * 5      # S = 5 x 2^254; sqrt(S) = 3.8e38, above binary32's largest number


def records(torch, values, rule):
    """(name, record) of the same elements through each norm call."""
    bits = bf16_bits(np.array(values, np.float32))
    rec = zs.ClipRecord()
    zs.GradNorm([on_gpu(torch, bits)], len(values), rule, rec)()
    yield "partials", rec
    rec = zs.ClipRecord()
    x = torch.tensor(values, dtype=torch.float32, device="cuda")
    zs.TensorsNorm(zs.TensorTable([x]), rule, rec)()
    yield "tensors", rec
    rec = zs.ClipRecord()
    zs.zs_clip_combine(x.double().square(), rule, rec)
    yield "sums", rec


@pytest.mark.parametrize("max_norm", [1.0, 3e38, math.inf])
@pytest.mark.parametrize("skip", [False, True])
def test_a_finite_sum_whose_root_binary32_cannot_hold(gpu, max_norm, skip):
    rule = zs.clip_rule(max_norm, 0.0, skip)
    limit = float(rule.max_norm)
    s, norm, coef = reference(np.array(BIG), limit, 0.0)
    assert math.isfinite(norm) and norm > F32_MAX and coef > 0
    for name, rec in records(gpu, BIG, rule):
        assert rec.sumsq.item() == s, name
        check(rec, s, norm, coef, 0 if skip else 1)
        assert rec.norm.item() == math.inf and rec.coef.item() > 0, name


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_infinite_and_nan_norms(gpu, bad):
    for max_norm in (0.0, 1.0, F32_MAX, math.inf):
        for skip in (False, True):
            for name, rec in records(gpu, [1.0, bad, 2.0], zs.clip_rule(max_norm, 0.0, skip)):
                want = bad if bad != bad else math.inf
                coef = math.nan if bad != bad else 1.0 if max_norm == math.inf else 0.0
                check(rec, want, want, coef, 0 if skip else 1)


def test_scaling_by_a_coefficient_of_an_unrepresentable_norm(gpu):
    """The elements are scaled by the record's coef where the rule does not skip,
    and keep every bit where it does."""
    torch = gpu
    for skip in (False, True):
        x = torch.tensor(BIG, dtype=torch.float32, device="cuda")
        table, rec = zs.TensorTable([x]), zs.ClipRecord()
        zs.TensorsNorm(table, zs.clip_rule(3e38, 0.0, skip), rec)()
        zs.zs_tensors_clip(table, rec)
        coef = np.float32(rec.coef.item())
        assert close(float(coef), float(np.float32(3e38)) / (math.sqrt(5) * 2.0 ** 127))
        want = np.array(BIG, np.float32) * (np.float32(1.0) if skip else coef)
        assert np.array_equal(x.cpu().numpy(), want)
