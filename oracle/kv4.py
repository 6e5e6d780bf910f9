"""4-bit K/V rows (oracle; test infrastructure only).

A row is 128 codes of 4 bits (sign, two exponent bits, one fraction bit) and
one e4m3 scale per 16 elements; an element stands for code * scale * global.
Written from that definition: the grids of the two small formats are listed
and a value goes to the nearest member, the one with an even bit pattern
between two. Only t = x * (1 / global) and max|t| / 6 are taken in fp32, as the
definition has them.
"""
import numpy as np

MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
#: e4m3 values >= 0 by bit pattern 0 .. 126 (127 is not a number)
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)]
                + [(1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(8, 127)])
NAN_SCALE = 127


def nearest_index(x, grid):
    """Index of the member of an ascending grid nearest to each x >= 0 (float64),
    the even index between two; past the last member, the last."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    take_hi = (up < down) | ((up == down) & (hi % 2 == 0))
    return np.where(take_hi, hi, lo)


def quantise(x, g):
    """Rows x [..., 128] (float32 values) -> codes uint8 [..., 128], scale bits uint8 [..., 8]."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(over="ignore", invalid="ignore"):
        t = (x * (np.float32(1) / np.float32(g))).astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    finite = np.isfinite(t).all(-1)
    t = np.where(finite[..., None], t, np.float32(0))
    s6 = (np.abs(t).max(-1) / np.float32(6)).astype(np.float32)
    scale = nearest_index(s6, E4M3).astype(np.uint8)
    s = E4M3[scale][..., None]
    y = np.abs(t.astype(np.float64)) / np.where(s > 0, s, 1.0)
    codes = np.where(s > 0, nearest_index(y, MAGNITUDES), 0).astype(np.uint8)
    codes |= ((t < 0) & (s > 0)).astype(np.uint8) << 3
    scale = np.where(finite, scale, np.uint8(NAN_SCALE)).astype(np.uint8)
    return codes.reshape(x.shape), scale


def pack(codes):
    """Codes [..., 128] -> bytes [..., 64]: the even element in the low half."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(packed, scale, g):
    """The float64 values that packed codes [..., 64] and scales [..., 8] stand for."""
    packed = np.asarray(packed, dtype=np.uint8)
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(*packed.shape[:-1], -1)
    v = MAGNITUDES[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.append(E4M3, np.nan)[np.asarray(scale) & 127]
    return v * np.repeat(s, 16, axis=-1) * float(np.float32(g))
