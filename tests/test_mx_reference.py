"""The microscaled formats' plain implementation, pinned by hand-computed values (CPU)."""
import numpy as np
import pytest

from tests import _mx_reference as ref


@pytest.mark.parametrize("fmt", ["fp4", "fp8"])
def test_every_code_is_its_own_nearest(fmt):
    values = ref.code_values(fmt)
    half = len(values) // 2
    for i, v in enumerate(values):
        if np.isnan(v):
            continue
        row = np.zeros((1, 32))
        row[0, 0], row[0, 1] = v, ref.SIZES[fmt][-1]    # the largest entry fixes the scale at 1
        codes, scales = ref.encode(row, fmt)
        assert scales[0, 0] == 127
        got = codes[0, 0] & 15 if fmt == "fp4" else codes[0, 0]
        assert got == (i if v != 0 or i < half else half)


def test_pins():
    row = np.zeros((1, 32))
    row[0, :8] = [4.0, 5.0, 7.0, 0.25, 0.75, -2.5, 3.5, -0.2]
    codes, scales = ref.encode(row, "fp4")              # scale 1, ties to even, 7 saturates
    assert scales[0, 0] == 127
    assert ref.decode(codes, scales, "fp4", 8).tolist() == [[4, 4, 6, 0, 1, -2, 4, -0.0]]
    row[0, :6] = [256.0, 500.0, 17.0, 19.0, 2.0 ** -10, -(2.0 ** -9) * 1.5]
    row[0, 6:] = 0
    codes, scales = ref.encode(row, "fp8")
    assert scales[0, 0] == 127
    assert ref.decode(codes, scales, "fp8", 6).tolist() == \
        [[256, 448, 16, 20, 0, -(2.0 ** -8)]]
    assert codes[0, :6].tolist() == [0x78, 0x7E, 0x58, 0x5A, 0, 0x82]


def test_scales_of_edges():
    x = np.zeros((7, 32))
    x[1, 3] = 1e-44                                     # below 2^-127 times the largest power
    x[2, 3] = np.float32(3.4e38)
    x[3, 3] = np.inf
    x[4, 3] = np.nan
    x[5, 3] = 8.0
    x[6, 3] = np.nextafter(8.0, 0)
    codes, scales = ref.encode(x, "fp4")
    assert scales[:, 0].tolist() == [0, 0, 252, 255, 255, 128, 127]
    assert not codes[[0, 3, 4]].any()
    assert np.isnan(ref.decode(codes, scales, "fp4", 32)[3:5]).all()
    assert ref.encode(x, "fp8")[1][:, 0].tolist() == [0, 0, 246, 255, 255, 122, 121]


def test_padding_and_rows():
    x = np.arange(70.0).reshape(2, 35)
    for fmt in ("fp4", "fp8"):
        codes, scales = ref.encode(x, fmt)
        assert codes.shape == (2, ref.row_bytes(fmt, 35)) and scales.shape == (2, 2)
        used = 3 if fmt == "fp8" else 2
        assert not codes[:, codes.shape[1] // 2 + used:].any()
        assert np.abs(ref.decode(codes, scales, fmt, 35) - x).max() <= 16


def test_bf16_round():
    assert ref.bf16_round([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, 1.0]).tolist() == \
        [1.0, 1 + 2.0 ** -6, 1.0]
