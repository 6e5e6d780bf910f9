"""Rotary positions with several axes (oracle; test infrastructure only).

Dims j and j + D/2 of a head turn by pos[axis(j)] * theta^(-2j/D). The axes
share the D/2 frequencies out in runs, or in turn while an axis has some left
of its section (what is left over goes to axis 0). float64.
"""
import numpy as np


def frequency_axes(half, sections, interleaved):
    if not interleaved:
        return np.repeat(np.arange(len(sections)), sections)
    n = len(sections)
    left = list(sections)
    out = []
    for j in range(half):
        a = j % n
        if a and left[a] > 0:
            left[a] -= 1
            out.append(a)
        else:
            out.append(0)
    return np.array(out)


def qk_norm_rope(x, w, pos, theta, sections=None, interleaved=False, eps=1e-6):
    """x (R, H, D), w (D,) or None, pos (axes, R) -> normed and turned rows (R, H, D)."""
    x = np.asarray(x, dtype=np.float64)
    D = x.shape[-1]
    half = D // 2
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    ax = frequency_axes(half, [half] if sections is None else sections, interleaved)
    ang = np.asarray(pos, dtype=np.float64)[ax].T * theta ** (-2.0 * np.arange(half) / D)
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)
