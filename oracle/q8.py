"""8-bit rows and their products (oracle; test infrastructure only).

A row is e4m3 codes and one scale that is a power of two; an element stands for
code * scale. Everything in float64 but for the residual's addition, which is
rounded as the residual stream is stored.
"""
import math

import numpy as np

#: The magnitudes of e4m3: (1 + f/8) 2^(e-7), and f/8 2^-6 where e is 0.
GRID = np.array([f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
                 for e in range(16) for f in range(8) if (e, f) != (15, 7)])


def nearest(x, grid=GRID):
    """The member of an ascending grid nearest to each |x|, signed; between two, the one of even index."""
    a = np.abs(np.asarray(x, dtype=np.float64))
    i = np.clip(np.searchsorted(grid, a), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (a - lo > hi - a) | ((a - lo == hi - a) & (i % 2 == 0))
    return np.copysign(np.where(up, hi, lo), x)


def code_values(codes):
    """The values of e4m3 codes (uint8), NaN for 0x7F and 0xFF."""
    b = np.asarray(codes, dtype=np.uint8)
    m = np.append(GRID, np.nan)[b & 127]
    return np.where(b > 127, -m, m)


def row_scale(top):
    """The least power of two with top <= 448 * it (1 for 0, NaN where top is not finite), at least 2^-126."""
    out = np.empty(np.shape(top))
    for i, t in np.ndenumerate(np.asarray(top, dtype=np.float64)):
        if not np.isfinite(t):
            out[i] = np.nan
        elif t == 0:
            out[i] = 1.0
        else:
            m, e = math.frexp(t / 448.0)  # t / 448 = m 2^e, 1/2 <= m < 1
            out[i] = 2.0 ** max(e - 1 if m == 0.5 else e, -126)
    return out


def quantise_rows(y):
    """(values, scales) of rows y [M][d] in 8 bits."""
    y = np.asarray(y, dtype=np.float64)
    scale = row_scale(np.abs(y).max(axis=1))
    with np.errstate(invalid="ignore"):
        return nearest(np.where(np.isfinite(scale)[:, None], y, 0) / scale[:, None]) * scale[:, None], scale


def norm_rows(s, weight, eps):
    """s / sqrt(mean s^2 + eps) * weight, row by row."""
    s = np.asarray(s, dtype=np.float64)
    y = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return y if weight is None else y * np.asarray(weight, dtype=np.float64)


def activate(v, act):
    if act == "silu":
        return v / (1 + np.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + np.vectorize(math.erf)(v / math.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v


def linear(x, w, bias=None, act="none", gated=False, residual=None):
    """act(x w^T + bias) + residual of values x [M][K], w [N][K] (gated: gate rows, then up rows); and the
    sums of the magnitudes |x| |w|^T that rounding errors of v are measured by, with v itself."""
    v, size = x @ w.T, np.abs(x) @ np.abs(w).T
    if bias is not None:
        v = v + bias
        size = size + np.abs(bias)
    n = w.shape[0] // 2 if gated else w.shape[0]
    out = activate(v[:, :n], act)
    if gated:
        out = out * v[:, n:]
    if residual is not None:
        out = out + residual
    return out, v, size
