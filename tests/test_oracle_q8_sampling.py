"""The oracle of 8-bit rows and of truncated sampling against their definitions."""
import itertools
import math

import numpy as np
import pytest
import torch

from oracle import q8
from oracle.sampling import gumbel_noise
from oracle.truncated_sampling import kept_tokens, sample_row


def test_grid_is_e4m3():
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(q8.code_values(np.arange(256)), codes, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 4001), np.linspace(-0.03, 0.03, 997), (q8.GRID[1:] + q8.GRID[:-1]) / 2])
    assert np.array_equal(q8.nearest(x), torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy())


def test_row_scale_is_the_least_power_of_two():
    for top in (448.0, 448.0000001, 224.0, 223.9, 1.0, 1e-30, 3e38, 447.99, 896.0, 1e-45):
        s = float(q8.row_scale(np.array([top]))[0])
        assert math.frexp(s)[0] == 0.5 and top <= 448 * s and (s == 2.0 ** -126 or top > 224 * s)
    assert q8.row_scale(np.array([0.0]))[0] == 1 and np.isnan(q8.row_scale(np.array([np.inf]))[0])


def test_quantised_rows_are_within_half_a_step():
    gen = np.random.default_rng(0)
    y = gen.standard_normal((7, 64)) * np.exp(gen.standard_normal((7, 1)) * 20)
    v, s = q8.quantise_rows(y)
    assert np.all(np.abs(v - y) <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * s[:, None]))
    assert np.array_equal(q8.quantise_rows(v)[0], v)


def test_linear_gated_matches_its_halves():
    gen = np.random.default_rng(1)
    x, w, b = gen.standard_normal((3, 8)), gen.standard_normal((10, 8)), gen.standard_normal(10)
    out, v, size = q8.linear(x, w, b, "silu", True)
    for m, n in itertools.product(range(3), range(5)):
        g = sum(x[m, k] * w[n, k] for k in range(8)) + b[n]
        u = sum(x[m, k] * w[n + 5, k] for k in range(8)) + b[n + 5]
        assert abs(out[m, n] - g / (1 + math.exp(-g)) * u) < 1e-12 and abs(v[m, n] - g) < 1e-12
    assert np.all(size >= np.abs(v) - 1e-12)


@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (3, 1.0, 0.0), (0, 0.7, 0.0), (0, 1.0, 0.2), (4, 0.8, 0.0), (5, 0.9, 0.1)])
def test_kept_tokens_by_their_definition(k, p, m):
    gen = np.random.default_rng(k + 7)
    for _ in range(50):
        l = np.round(gen.standard_normal(9) * 2) / 2  # with ties
        mask, _ = kept_tokens(l, 0.7, k, p, m)
        r = float(np.float32(1) / np.float32(0.7))
        w = {v: math.exp((l[v] - l.max()) * r) for v in range(9)}
        order = sorted(range(9), key=lambda v: (-l[v], v))
        keep = [v for v in (order[:k] if k else order) if not m or w[v] >= float(np.float32(m))] or order[:1]
        if p < 1:
            total, have, n = sum(w[v] for v in keep), 0.0, 0
            while have < float(np.float32(p)) * total:
                have += w[keep[n]]
                n += 1
            keep = keep[:n]
        assert sorted(np.flatnonzero(mask)) == sorted(keep)


def test_sample_row_is_a_draw_from_the_kept_distribution():
    l = np.array([2.0, 1.0, 1.5, -1.0, 0.5, -np.inf, 2.0, 0.0])
    n = 20000
    mask, _ = kept_tokens(l, 1.3, 5, 0.9, 0.0)
    want = np.where(mask, np.exp(l / 1.3), 0)
    want /= want.sum()
    got = np.bincount([sample_row(l, 11, pos, 2, 1.3, 5, 0.9)[0] for pos in range(n)], minlength=8) / n
    # five standard deviations of a frequency
    assert np.all(np.abs(got - want) <= 5 * np.sqrt(want * (1 - want) / n))
    token, gap, _ = sample_row(l, 3, 9, 1, temperature=0)
    assert token == 0 and gap == 0
    z = l + gumbel_noise(3, 1, 9, 8)
    assert sample_row(l, 3, 9, 1)[0] == int(np.argmax(z))
