"""Pins of the oracle for 4-bit rows and multi-axis rotary positions (CPU)."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import dense, kv4, rope


def test_e4m3_grid_is_torchs():
    bits = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(kv4.E4M3, bits.view(torch.float8_e4m3fn).double().numpy())
    assert torch.tensor([127], dtype=torch.uint8).view(torch.float8_e4m3fn).isnan().all()


def test_scale_rounding_is_torchs():
    x = np.abs(W.rng(1).standard_normal(20000).astype(np.float32)) * np.exp2(W.rng(2).uniform(-14, 8.5, 20000)).astype(np.float32)
    x = np.minimum(x, np.float32(448))
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(kv4.nearest_index(x, kv4.E4M3), want)


def test_code_is_the_nearest_of_the_sixteen_and_ties_go_to_the_even_one():
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 9.0: 7}
    for x, c in ties.items():
        assert kv4.nearest_index(x, kv4.MAGNITUDES) == c
    y = np.linspace(0, 7, 4001)
    i = kv4.nearest_index(y, kv4.MAGNITUDES)
    assert np.array_equal(np.abs(kv4.MAGNITUDES[i] - y), np.abs(kv4.MAGNITUDES[None] - y[:, None]).min(1))


@pytest.mark.parametrize("g", [1.0, 0.25, 6.1 / 2688])
def test_a_row_comes_back_within_half_a_step_of_its_group(g):
    x = W.bf16_bits_to_f32(W.normal_bf16(W.rng(3), (50, 128)))
    codes, scale = kv4.quantise(x, g)
    v = kv4.values(kv4.pack(codes), scale, g)
    amax = np.repeat(np.abs(x).reshape(50, 8, 16).max(-1), 16, axis=-1)
    # the widest step is 2 of 6; the scale's rounding (half a step, 2^-4) moves both the grid and the largest value
    assert np.all(np.abs(v - x) <= amax * (1 / 6 + 2 ** -4 + 1e-6))


def test_quantising_values_of_the_form_gives_them_back():
    x = kv4.values(W.rng(4).integers(0, 256, (20, 64)).astype(np.uint8), np.full((20, 8), 0x38, np.uint8), 1.0)
    x[:, ::16] = 6.0  # the group's scale is 1
    codes, scale = kv4.quantise(x, 1.0)
    assert np.array_equal(kv4.values(kv4.pack(codes), scale, 1.0), x) and np.all(scale == 0x38)


def test_zero_tiny_huge_and_not_finite_groups():
    x = np.zeros((1, 128), np.float32)
    x[0, 16:32] = 1e-4        # / 6 is under half the least scale: the group is zero
    x[0, 32:48] = 1e6         # over 6 * 448
    x[0, 48] = np.nan
    x[0, 64] = -np.inf
    codes, scale = kv4.quantise(x, 1.0)
    assert scale[0].tolist() == [0, 0, 126, 127, 127, 0, 0, 0]
    v = kv4.values(kv4.pack(codes), scale, 1.0)[0]
    assert np.all(v[:32] == 0) and np.all(v[32:48] == 2688) and np.isnan(v[48:80]).all() and np.all(v[80:] == 0)


def test_one_axis_is_the_layers_rope_and_norm():
    x = W.rng(5).standard_normal((7, 3, 128))
    w = W.rng(6).uniform(0.5, 1.5, 128)
    pos = W.rng(7).integers(0, 5000, 7)
    want = dense.rope(dense.rmsnorm(x, w, 1e-6), pos, 1e6)
    np.testing.assert_allclose(rope.qk_norm_rope(x, w, pos[None], 1e6), want, rtol=0, atol=1e-9)


def test_equal_positions_on_every_axis_are_one_axis():
    x = W.rng(8).standard_normal((5, 2, 64))
    pos = W.rng(9).integers(0, 5000, 5)
    one = rope.qk_norm_rope(x, None, pos[None], 1e4)
    for sec, il in (([16, 8, 8], False), ([16, 8, 8], True), ([24, 8], True)):
        np.testing.assert_allclose(rope.qk_norm_rope(x, None, np.stack([pos] * len(sec)), 1e4, sec, il), one, atol=1e-12)


def test_frequency_axes():
    assert rope.frequency_axes(6, [2, 3, 1], False).tolist() == [0, 0, 1, 1, 1, 2]
    assert rope.frequency_axes(8, [4, 2, 2], True).tolist() == [0, 1, 2, 0, 1, 2, 0, 0]
    a = rope.frequency_axes(64, [24, 20, 20], True)
    assert [(a == i).sum() for i in range(3)] == [24, 20, 20] and a[:6].tolist() == [0, 1, 2, 0, 1, 2]
