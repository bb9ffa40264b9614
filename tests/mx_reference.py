"""A plain restatement, in 64-bit floats and integers on the host, of microscaled 4-bit matrices: their codes, scale bytes
and values."""

import numpy as np

GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def quantize(x):
    """(codes rows x k_p, scale bytes rows x k_p / 32) of a float64 matrix, k_p = k rounded up to 32."""
    rows, k = x.shape
    blocks = -(-k // 32)
    t = np.zeros((rows, blocks * 32))
    t[:, :k] = x
    t = t.reshape(rows, blocks, 32)
    most = np.abs(t).max(2)  # NaN where one is
    bad = ~np.isfinite(most)
    exponent = np.frexp(np.where(bad, 1.0, most))[1] - 1  # floor(log2); of 0: -1
    exponent = np.where(most == 0, -10000, exponent)
    e = np.maximum(exponent - 2, -127)
    a = np.abs(np.where(bad[:, :, None], 0.0, t)) * np.exp2(-e.astype(np.float64))[:, :, None]
    codes = np.zeros(a.shape, dtype=np.int64)
    for c in range(1, 8):  # past the middle of c - 1 and c; on it, to the even one
        middle = (GRID[c - 1] + GRID[c]) / 2
        codes += (a >= middle) if c % 2 == 0 else (a > middle)
    codes += 8 * np.signbit(t)
    codes = np.where(bad[:, :, None], 0, codes)
    return codes.reshape(rows, -1), np.where(bad, 255, e + 127)


def values(codes, scales):
    """The float64 values of unpacked codes and scale bytes."""
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    return v * np.repeat(s, 32, axis=1)


def pack(codes, scales, rows, k):
    """The two arrays as the library lays them out."""
    packed = (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)
    tiles = np.full((-(-rows // 128), -(-k // 256), 1024), 127, dtype=np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(scales.shape[1]), indexing="ij")
    tiles[r // 128, b // 8, b % 8 // 4 * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4] = scales
    return packed, tiles
