"""Plain implementation of the microscaled formats in 64 bits (numpy): codes,
scales, quantisation by the nearest entry of the format's table, and products."""
import numpy as np

BLOCK = 32
FP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
FP8 = np.array([i / 512.0 for i in range(8)] +
               [(1 + i / 8.0) * 2.0 ** e for e in range(-6, 9) for i in range(8)][:-1])
SIZES = {"fp4": FP4, "fp8": FP8}
TOP = {"fp4": 2, "fp8": 8}


def row_bytes(fmt, cols):
    return -(-cols // BLOCK) * (16 if fmt == "fp4" else 32)


def code_values(fmt):
    """The value of every code."""
    sizes = SIZES[fmt] if fmt == "fp4" else np.append(FP8, np.nan)
    return np.concatenate((sizes, -sizes))


def decode(codes, scales, fmt, cols):
    """float64 [rows, cols] of codes [rows, bytes] and scales [rows, blocks]."""
    if fmt == "fp4":
        codes = np.stack((codes & 15, codes >> 4), axis=2).reshape(codes.shape[0], codes.shape[1] * 2)
    factor = np.exp2(np.arange(256.0) - 127)
    factor[255] = np.nan
    each = np.repeat(factor[scales], BLOCK, axis=1)
    return (code_values(fmt)[codes] * each)[:, :cols]


def encode(x, fmt):
    """(codes, scales) of a float64 matrix [rows, cols]."""
    x = np.asarray(x, np.float64)
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    full = np.zeros((rows, nb * BLOCK))
    full[:, :cols] = x
    full = full.reshape(rows, nb, BLOCK)
    finite = np.isfinite(full).all(axis=2)
    peak = np.abs(np.where(finite[..., None], full, 0)).max(axis=2, initial=0)
    e = np.frexp(np.where(peak > 0, peak, 1.0))[1] - 1 - TOP[fmt]
    b = np.where(peak > 0, np.maximum(e, -127) + 127, 0)
    size = np.abs(full) / np.exp2(b - 127.0)[..., None]
    size[~finite] = 0
    table = SIZES[fmt]
    between = (table[1:] + table[:-1]) / 2
    place = np.searchsorted(between, size)            # ties stay at the lower entry
    tie = between[np.minimum(place, len(between) - 1)] == size
    place = np.minimum(np.where(tie & (place % 2 == 1), place + 1, place), len(table) - 1)
    sign = np.signbit(full) & finite[..., None]
    code = (place + np.where(sign, 8 if fmt == "fp4" else 128, 0)).astype(np.uint8)
    code = code.reshape(rows, nb * BLOCK)
    if fmt == "fp4":
        code = code[:, 0::2] | (code[:, 1::2] << 4)
    return np.ascontiguousarray(code), np.where(finite, b, 255).astype(np.uint8)


def bf16_round(x):
    """float64 values rounded to the nearest bf16, ties to even, as float32.  Exact for
    finite float64 inputs whose float32 is exact or not a tie of bf16."""
    x32 = np.asarray(x, np.float64).astype(np.float32)
    u = x32.view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> np.uint64(16)) & np.uint64(1))) & np.uint64(0xFFFF0000))
    return r.astype(np.uint32).view(np.float32)
