"""The norm and clipping calls on the CPU: how a list of tensors is cut into
pieces, what each call refuses (the arguments are checked before the state of
the library, so a call that passes every check ends in "not initialized"), and
the binding's own checks.  No call gets as far as a device."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest

import sharded_mixed_precision_shard_amd as zs
from tests.conftest import ROOT
from tests.test_binding_checks import FakeGpuTensor

PIECE = 8192
SIZE = {0: 2, 1: 2, 2: 4}
INVALID, MISALIGNED, ALIASING, NOT_INIT = (zs.ZS_ERR_INVALID_ARGUMENT, zs.ZS_ERR_MISALIGNED,
                                           zs.ZS_ERR_ALIASING, zs.ZS_ERR_NOT_INITIALIZED)
HOLE = 1 << 40   # addresses far from the others


def test_struct_layouts_and_constants_match_the_header():
    src = r'''
    #include <stddef.h>
    #include <stdio.h>
    #include "zs.h"
    int main(void) {
      printf("%zu %zu %zu %zu %zu ", sizeof(zs_clip), sizeof(zs_clip_rule), sizeof(zs_tensor),
             sizeof(zs_piece), sizeof(zs_tensor_table));
      printf("%zu %zu %zu %zu %zu ", offsetof(zs_clip, norm), offsetof(zs_clip, coef),
             offsetof(zs_clip, apply), offsetof(zs_tensor, dtype), offsetof(zs_piece, n));
      printf("%d %d %d %d %d\n", ZS_NORM_WORKSPACE_BYTES, ZS_MAX_SUMS, ZS_DTYPE_BF16,
             ZS_DTYPE_FP16, ZS_DTYPE_FP32);
      return 0; }
    '''
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "probe.c"), os.path.join(d, "probe")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), "-o", exe, c],
                       check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True,
                                              check=True).stdout.split()]
    assert got == [ctypes.sizeof(zs.ZsClip), ctypes.sizeof(zs.ZsClipRule),
                   ctypes.sizeof(zs.ZsTensor), ctypes.sizeof(zs.ZsPiece),
                   ctypes.sizeof(zs.ZsTensorTable), zs.ZsClip.norm.offset, zs.ZsClip.coef.offset,
                   zs.ZsClip.apply.offset, zs.ZsTensor.dtype.offset, zs.ZsPiece.n.offset,
                   zs.ZS_NORM_WORKSPACE_BYTES, zs.ZS_MAX_SUMS, zs.ZS_DTYPE["torch.bfloat16"],
                   zs.ZS_DTYPE["torch.float16"], zs.ZS_DTYPE["torch.float32"]]


@pytest.mark.parametrize("seed", range(8))
def test_pieces_cover_every_tensor_once_and_start_aligned(seed):
    rng = np.random.default_rng(seed)
    tensors, at = [], 1 << 30
    for _ in range(int(rng.integers(1, 60))):
        dtype = int(rng.integers(0, 3))
        n = int(rng.choice([0, 1, 2, 7, 64, 2047, 4096, 4097, 20000, 100003]))
        at += int(rng.integers(0, 5000))
        at += -at % SIZE[dtype]
        tensors.append((at, n, dtype))
        at += n * SIZE[dtype]
    pieces = [(p.addr, p.n, p.dtype) for p in zs.zs_tensor_pieces(tensors)]
    it = iter(pieces)
    for addr, n, dtype in tensors:
        a, left = addr, n
        while left:
            pa, pn, pd = next(it)
            assert (pa, pd) == (a, dtype) and 0 < pn <= left
            assert pa // PIECE == (pa + pn * SIZE[pd] - 1) // PIECE   # inside one stretch
            if a != addr:
                assert pa % PIECE == 0
            a, left = a + pn * SIZE[pd], left - pn
        assert a == addr + n * SIZE[dtype]
    assert next(it, None) is None


def test_pieces_of_nothing():
    assert len(zs.zs_tensor_pieces([])) == 0
    assert len(zs.zs_tensor_pieces([(0, 0, 0), (0, 0, 2)])) == 0


def _pieces_status(tensors, count=None):
    try:
        zs.zs_tensor_pieces(tensors)
    except zs.ZsError as e:
        return e.status
    return zs.ZS_OK


def test_pieces_refusals():
    a = 1 << 30
    assert _pieces_status([(a, 100, 0), (a + 200, 100, 0)]) == zs.ZS_OK   # they touch
    assert _pieces_status([(a, 100, 0), (a, 100, 0)]) == ALIASING         # one listed twice
    assert _pieces_status([(a + 198, 5, 0), (a, 100, 0)]) == ALIASING     # by one element
    assert _pieces_status([(a, 1000, 2), (a + 400, 1, 1)]) == ALIASING    # one inside another
    assert _pieces_status([(a, 10 ** 6, 2), (a + 4, 1, 2), (a + 10 ** 7, 4, 2)]) == ALIASING
    assert _pieces_status([(a, 100, 0), (a + 2, 0, 0)]) == zs.ZS_OK       # an empty one inside
    assert _pieces_status([(a + 1, 4, 0)]) == MISALIGNED
    assert _pieces_status([(a + 2, 4, 2)]) == MISALIGNED
    assert _pieces_status([(a + 2, 4, 1)]) == zs.ZS_OK
    assert _pieces_status([(a, -1, 0)]) == INVALID
    assert _pieces_status([(0, 1, 0)]) == INVALID
    assert _pieces_status([(a, 1, 3)]) == INVALID and _pieces_status([(a, 1, -1)]) == INVALID
    assert _pieces_status([(2 ** 64 - 8, 8, 2)]) == INVALID               # past the address space
    lib = zs.load_library()
    one, made = (zs.ZsTensor * 1)(zs.ZsTensor(a, 10 * PIECE, 2, 0)), ctypes.c_int64(-1)
    out = (zs.ZsPiece * 39)()
    assert lib.zs_tensor_pieces(one, 1, out, 39, ctypes.byref(made)) == INVALID
    assert made.value == 40                                               # what it would take
    assert lib.zs_tensor_pieces(one, 1, None, 0, None) == INVALID
    assert lib.zs_tensor_pieces(None, 1, None, 0, ctypes.byref(made)) == INVALID
    assert lib.zs_tensor_pieces(one, -1, None, 0, ctypes.byref(made)) == INVALID
    # a size no device holds is counted, not walked
    one[0].n = 1 << 59
    assert lib.zs_tensor_pieces(one, 1, None, 0, ctypes.byref(made)) == zs.ZS_OK
    assert made.value == 1 << 48
    assert lib.zs_tensor_pieces(one, 1, out, 39, ctypes.byref(made)) == INVALID
    assert made.value == 1 << 48
    assert lib.zs_tensor_pieces(one, 1, out, -1, ctypes.byref(made)) == INVALID
    one[0].n, one[0].reserved = 10 * PIECE, 1
    assert lib.zs_tensor_pieces(one, 1, None, 0, ctypes.byref(made)) == INVALID


def _norm(grads=(4096, 8192), k=None, n=1000, scale=1.0, rule=None, clip=HOLE,
          ws=HOLE + (1 << 20), scales=None):
    lib = zs.load_library()
    gp = (ctypes.c_void_p * max(len(grads or ()), 1))(*(grads or ()))
    g = ctypes.cast(gp, ctypes.c_void_p) if grads is not None else None
    k = len(grads) if k is None else k
    r = None if rule is None else ctypes.byref(rule)
    if scales is None:
        return lib.zs_grad_norm(g, k, n, scale, r, clip, ws, None)
    sp = (ctypes.c_void_p * max(len(scales), 1))(*scales)
    return lib.zs_grad_norm_q8grad(g, ctypes.cast(sp, ctypes.c_void_p), k, n, scale, r, clip, ws,
                                   None)


def test_norm_refusals():
    assert _norm() == NOT_INIT                       # every argument is fine
    assert _norm(n=0, grads=(), k=1) == NOT_INIT     # no elements: no partial is looked at
    assert _norm(k=0) == INVALID and _norm(k=17) == INVALID
    assert _norm(n=-1) == INVALID and _norm(n=2 ** 63 - 1) == INVALID
    assert _norm(grads=None, k=1) == INVALID
    assert _norm(grads=(4096, 0)) == INVALID
    assert _norm(grads=(4096, 8200)) == MISALIGNED
    for bad in (float("inf"), float("nan")):
        assert _norm(scale=bad) == INVALID
    assert _norm(clip=None) == INVALID and _norm(ws=None) == INVALID
    assert _norm(clip=HOLE + 4) == MISALIGNED and _norm(ws=HOLE + (1 << 20) + 4) == MISALIGNED
    # the record and the workspace: apart from each other and from every partial
    assert _norm(clip=HOLE, ws=HOLE + 16) == ALIASING
    assert _norm(clip=HOLE, ws=HOLE - zs.ZS_NORM_WORKSPACE_BYTES + 8) == ALIASING
    assert _norm(clip=HOLE, ws=HOLE + 24) == NOT_INIT
    assert _norm(clip=8192 + 1992) == ALIASING       # the last elements of partial 1
    assert _norm(grads=(4096, HOLE + (1 << 20) + 64)) == ALIASING
    # int8: codes 16-byte, scales 4-byte aligned, both given
    assert _norm(scales=(1 << 20, 1 << 21)) == NOT_INIT
    assert _norm(scales=(1 << 20, 0)) == INVALID
    assert _norm(scales=(1 << 20, (1 << 21) + 2)) == MISALIGNED
    assert _norm(scales=(1 << 20, HOLE + 20)) == ALIASING


def test_rule_refusals():
    for rule in (zs.clip_rule(-1.0), zs.clip_rule(float("nan")), zs.clip_rule(1.0, eps=-1e-6),
                 zs.clip_rule(1.0, eps=float("nan")), zs.clip_rule(1.0, eps=float("inf")),
                 zs.ZsClipRule(1.0, 0.0, 0, 1)):
        assert _norm(rule=rule) == INVALID
        assert zs.load_library().zs_clip_combine(4096, 1, ctypes.byref(rule), HOLE, None) == INVALID
    for rule in (zs.clip_rule(0.0), zs.clip_rule(float("inf")), zs.clip_rule(1.0, 0.0, True)):
        assert _norm(rule=rule) == NOT_INIT


def test_combine_refusals():
    f = zs.load_library().zs_clip_combine
    assert f(4096, 8, None, HOLE, None) == NOT_INIT
    assert f(HOLE, 1, None, HOLE, None) == NOT_INIT   # the record's own sum
    assert f(HOLE, 2, None, HOLE, None) == ALIASING
    assert f(HOLE + 8, 1, None, HOLE, None) == ALIASING
    assert f(HOLE - 8, 2, None, HOLE, None) == ALIASING
    assert f(None, 1, None, HOLE, None) == INVALID and f(4096, 1, None, None, None) == INVALID
    assert f(4096, 0, None, HOLE, None) == INVALID
    assert f(4096, zs.ZS_MAX_SUMS + 1, None, HOLE, None) == INVALID
    assert f(4100, 1, None, HOLE, None) == MISALIGNED
    assert f(4096, 1, None, HOLE + 4, None) == MISALIGNED


def test_table_refusals():
    lib = zs.load_library()

    def table(pieces=4096, count=10):
        return ctypes.byref(zs.ZsTensorTable(pieces, count))
    ws = HOLE + (1 << 20)
    assert lib.zs_tensors_norm(table(), None, HOLE, ws, None) == NOT_INIT
    assert lib.zs_tensors_norm(table(0, 0), None, HOLE, ws, None) == NOT_INIT
    assert lib.zs_tensors_clip(table(), HOLE, None) == NOT_INIT
    for t, want in ((None, INVALID), (table(0, 1), INVALID), (table(4096, -1), INVALID),
                    (table(4104), MISALIGNED)):
        assert lib.zs_tensors_norm(t, None, HOLE, ws, None) == want
        assert lib.zs_tensors_clip(t, HOLE, None) == want
    assert lib.zs_tensors_norm(table(HOLE), None, HOLE, ws, None) == ALIASING
    assert lib.zs_tensors_norm(table(ws), None, HOLE, ws, None) == ALIASING
    assert lib.zs_tensors_norm(table(), None, None, ws, None) == INVALID
    assert lib.zs_tensors_norm(table(), None, HOLE, None, None) == INVALID
    assert lib.zs_tensors_clip(table(), None, None) == INVALID
    assert lib.zs_tensors_clip(table(), HOLE + 4, None) == MISALIGNED


def test_clipped_step_refusals():
    """The record and the buffers are looked at first, then what every step checks
    (on this machine: that the library is initialized)."""
    lib, hp = zs.load_library(), zs.hparams()
    b, st = zs.ZsStepBuffers(), zs.ZsSegTable(4096, 1, 0)

    def call(buffers=b, clip=HOLE):
        return lib.zs_shard_step_clipped(0, ctypes.byref(buffers) if buffers else None, 1, 100,
                                         ctypes.byref(st), ctypes.byref(hp), 1, 0, clip, None)
    assert call() == NOT_INIT
    assert call(buffers=None) == INVALID and call(clip=None) == INVALID


class Tensor:
    """Answers what the binding asks of a GPU tensor, at an address never used."""

    def __init__(self, shape, strides, dtype="torch.bfloat16", addr=1 << 30, index=0):
        import torch
        self.shape, self._strides, self.dtype, self._a = shape, strides, dtype, addr
        self.is_cuda, self.device = True, torch.device("cuda", index)

    def stride(self):
        return self._strides

    def is_contiguous(self):
        want = 1
        for s, n in reversed(list(zip(self._strides, self.shape))):
            if n != 1 and s != want:
                return False
            want *= n
        return True

    def data_ptr(self):
        return self._a

    def numel(self):
        return int(np.prod(self.shape, dtype=np.int64))


def test_binding_takes_dense_tensors_in_any_order():
    pytest.importorskip("torch")
    for shape, strides in (((6, 4), (4, 1)), ((4, 6), (1, 4)), ((2, 3, 4), (1, 8, 2)),
                           ((5, 1, 2), (2, 99, 1)), ((), ())):
        p = zs.zs_tensor_pieces([Tensor(shape, strides)])
        assert sum(x.n for x in p) == int(np.prod(shape, dtype=np.int64))
    for shape, strides in (((6, 4), (8, 1)), ((6, 4), (0, 1)), ((4,), (2,)), ((3, 3), (1, 1))):
        with pytest.raises(ValueError, match="dense"):
            zs.zs_tensor_pieces([Tensor(shape, strides)])
    with pytest.raises(TypeError, match="float64"):
        zs.zs_tensor_pieces([Tensor((4,), (1,), "torch.float64")])
    torch = pytest.importorskip("torch")
    with pytest.raises(ValueError, match="GPU tensor"):
        zs.zs_tensor_pieces([torch.zeros(4)])


def test_binding_refusals_of_the_clipped_step():
    n = 1000
    f = [FakeGpuTensor(4 * n) for _ in range(3)] + [FakeGpuTensor(2 * n)]
    g, st, hp, rec = [FakeGpuTensor(2 * n)], zs.seg_table(FakeGpuTensor(16), 1), zs.hparams(), \
        FakeGpuTensor(24)
    with pytest.raises(ValueError, match="needs a record"):
        zs.zs_shard_step_clipped("base", *f, g, n, st, hp, 1, None)
    with pytest.raises(ValueError, match="clip holds"):
        zs.ShardStep(*f, g, n, st, hp, clip=FakeGpuTensor(16))
    with pytest.raises(TypeError, match="host"):
        zs.ShardStep(*f, g, n, st, hp, clip=np.zeros(24, np.uint8))
    with pytest.raises(ValueError, match="no launch cfg"):
        zs.ShardStep(*f, g, n, st, hp, cfg=dict(chunk_tiles=2), clip=rec)
    with pytest.raises(ValueError, match="m holds"):
        zs.zs_shard_step_clipped("base", f[0], FakeGpuTensor(2 * n), f[2], f[3], g, n, st, hp, 1, rec)
    # every form takes exactly the buffers it names (null addresses: the library refuses)
    nb = -(-n // 256)
    more = dict(q8ag=dict(param_q8=FakeGpuTensor(n), param_q8_scale=FakeGpuTensor(4 * nb)),
                q8grad=dict(qscales=[FakeGpuTensor(4 * nb)]))
    for form in zs.ZS_VARIANT:
        state = FakeGpuTensor(4 * zs.packed_floats(n))
        head = (state, None, None, f[3]) if form.startswith("packed") else f
        kw = {k: v for name, v in more.items() if form.endswith(name) for k, v in v.items()}
        if form.endswith("_sr"):
            kw["seed"] = 3
        step = zs.ShardStep(*head, g, n, st, hp, variant=form, clip=rec, **kw)
        assert step(1, check=False) in (NOT_INIT, INVALID)


def test_binding_refusals():
    torch = pytest.importorskip("torch")
    n = 1000
    g, ws, rec = [FakeGpuTensor(2 * n)] * 2, FakeGpuTensor(zs.ZS_NORM_WORKSPACE_BYTES), \
        FakeGpuTensor(24)
    with pytest.raises(ValueError, match="k=3 but 2 grads"):
        zs.zs_grad_norm(g, 3, n, 1.0, None, rec, ws)
    with pytest.raises(ValueError, match=r"grads\[1\] holds"):
        zs.zs_grad_norm([g[0], FakeGpuTensor(2 * n - 2)], 2, n, 1.0, None, rec, ws)
    with pytest.raises(ValueError, match="clip holds"):
        zs.zs_grad_norm(g, 2, n, 1.0, None, FakeGpuTensor(16), ws)
    with pytest.raises(ValueError, match="workspace holds"):
        zs.zs_grad_norm(g, 2, n, 1.0, None, rec, FakeGpuTensor(1024))
    with pytest.raises(TypeError, match="ZsClipRule"):
        zs.zs_grad_norm(g, 2, n, 1.0, 1.0, rec, ws)
    with pytest.raises(ValueError, match="1 qscales for 2 partials"):
        zs.zs_grad_norm_q8grad(g, [FakeGpuTensor(16)], 2, n, 1.0, None, rec, ws)
    with pytest.raises(ValueError, match=r"qscales\[1\] holds"):
        zs.zs_grad_norm_q8grad(g, [FakeGpuTensor(16), FakeGpuTensor(12)], 2, n, 1.0, None, rec, ws)
    with pytest.raises(ValueError, match="GPU tensor"):
        zs.zs_clip_combine(torch.zeros(2, dtype=torch.float64), None, rec)
    with pytest.raises(TypeError, match="float64"):
        zs.zs_clip_combine(torch.zeros(2), None, rec)
    with pytest.raises(ValueError, match="different devices"):
        zs.TensorTable([Tensor((4,), (1,)), Tensor((4,), (1,), addr=1 << 31, index=1)])
