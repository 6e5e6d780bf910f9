"""Sampling with temperature, top-k, min-p and top-p (oracle; test
infrastructure only): "Vision Is Not Overhead ..." (arXiv 2609.00355), Section
5.4, the committed token is a draw from the target's own verified row. The noise
is that of sampling.py. Everything in float64 but 1 / T, which is fp32.
"""
import numpy as np

from .sampling import gumbel_noise


def kept_tokens(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(mask of what is kept, how near a token came to top_p's border or a weight to min_p, relatively)."""
    l = np.asarray(logits, dtype=np.float64)
    V = l.size
    r = float(np.float32(1) / np.float32(temperature))
    order = np.lexsort((np.arange(V), -l))
    with np.errstate(invalid="ignore"):
        w = np.exp((l[order] - l[order[0]]) * r)
    n = V if top_k <= 0 else min(int(top_k), V)
    n = min(n, int((w > 0).sum()))
    near = np.inf
    if min_p > 0:
        m = float(np.float32(min_p))
        near = np.abs(w[1:] - m).min(initial=np.inf) / m
        n = min(n, max(1, int((w >= m).sum())))
    if top_p < 1:
        upto = np.cumsum(w[:n])
        target = max(float(np.float32(top_p)), 0.0) * upto[-1]
        near = min(near, np.abs(upto - target).min() / upto[-1])
        n = max(1, int((upto < target).sum()) + 1)
    mask = np.zeros(V, dtype=bool)
    mask[order[:n]] = True
    return mask, near


def sample_row(logits, seed, pos, seq=0, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, gap, near): the draw, best minus second best, and kept_tokens' near."""
    l = np.asarray(logits, dtype=np.float64)
    if temperature == 0:
        z, near = l.copy(), np.inf
    else:
        mask, near = kept_tokens(l, temperature, top_k, top_p, min_p)
        z = l * float(np.float32(1) / np.float32(temperature)) + gumbel_noise(seed, seq, pos, l.size)
        z[~mask] = -np.inf
    token = int(np.argmax(z))
    rest = np.delete(z, token).max()
    return token, (z[token] - rest if np.isfinite(rest) else np.inf), near
