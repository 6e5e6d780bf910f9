"""Rows into 4-bit caches and back: every byte equals the oracle's, nothing
else of the cache changes, and the values read are the bytes' values."""
import numpy as np
import pytest
import torch

import workloads as W
from _kv4_util import bytes_of, layer_of, up
from _util import bf16_tensor
from oracle import kv4 as okv4

pytestmark = pytest.mark.gpu


def fresh(gen, n_layers, Hkv, slots):
    u8 = lambda *s: gen.integers(0, 256, s).astype(np.uint8)
    return [[u8(Hkv, slots, 64), u8(Hkv, slots, 8), u8(Hkv, slots, 64), u8(Hkv, slots, 8)] for _ in range(n_layers)]


# (layers, kv heads, T, rows, slots, t_cap): one row, odd rows, a full block of 128 and one past it, a gap between heads, T = 0
SHAPES = [(1, 1, 0, 1, 2, 2), (2, 3, 5, 7, 20, 20), (1, 2, 127, 128, 258, 255), (36, 8, 17, 64, 90, 81), (1, 2, 1, 129, 200, 130),
          (49, 1, 0, 3, 4, 4), (128, 2, 9, 2, 30, 11)]


@pytest.mark.parametrize("n_layers,Hkv,T,rows,slots,t_cap", SHAPES)
@pytest.mark.parametrize("kg,vg", [(1.0, 0.125), (6.1 / 2688, 0.3)])
def test_rows_land_quantised_at_T_and_come_back(dev, clean_status, n_layers, Hkv, T, rows, slots, t_cap, kg, vg):
    import tree_verified_block_gb300 as g
    gen = W.rng(n_layers, rows, T)
    host = fresh(gen, n_layers, Hkv, slots)
    src = W.normal_bf16(gen, (n_layers, 2, Hkv, rows, 128), 1.5)
    t_len = torch.tensor([T], dtype=torch.int32, device=dev)
    layers = [layer_of(g, h, t_len, dev, kg, vg, t_cap) for h in host]
    g.kv4_write_rows(bf16_tensor(src, dev), layers, rows)
    dst = torch.full((n_layers, 2, Hkv, rows, 128), 77.0, dtype=torch.bfloat16, device=dev)
    g.kv4_read_rows(g.Views(layers), T, rows, dst)
    x = W.bf16_bits_to_f32(src)
    got_rows = dst.double().cpu().numpy()
    for l in range(n_layers):
        want = [a[:, :t_cap].copy() for a in host[l]]
        for i, gl in ((0, kg), (1, vg)):
            codes, scale = okv4.quantise(x[l, i], gl)
            want[2 * i][:, T:T + rows], want[2 * i + 1][:, T:T + rows] = okv4.pack(codes), scale
            v = okv4.values(okv4.pack(codes), scale, gl)
            # scale * global and the product are rounded to fp32 (2^-24 each), the result to bf16 (2^-8)
            assert np.all(np.abs(got_rows[l, i] - v) <= np.abs(v) * (2 ** -8 + 2 ** -22))
        for a, b in zip(bytes_of(layers[l]), want):
            assert np.array_equal(a, b), l
    assert int(t_len) == T


def test_every_bf16_pattern_and_mixed_groups(dev, clean_status):
    """All 65536 bf16 patterns, alone in a group and next to others: ties, subnormals, infinities, NaN."""
    import tree_verified_block_gb300 as g
    pat = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    mixed = W.rng(3).permutation(pat).reshape(512, 128)
    near = ((127 + W.rng(4).integers(-4, 5, (512, 128))) << 7 | W.rng(5).integers(0, 128, (512, 128))).astype(np.uint16)
    alone = np.zeros((8192, 128), np.uint16)
    alone[:, ::16] = pat.reshape(8192, 8)
    src = np.concatenate([mixed, near, alone])[None, None].repeat(2, 1)[:, :, None]
    rows = src.shape[3]
    t_len = torch.zeros(1, dtype=torch.int32, device=dev)
    for kg, vg in ((1.0, 3.0), (1 / 448, 2.0 ** -20)):
        layer = g.KV4Layer.empty(1, rows, t_len, kg, vg, dev)
        g.kv4_write_rows(bf16_tensor(src, dev), [layer], rows)
        got = bytes_of(layer)
        x = W.bf16_bits_to_f32(src)
        for i, gl in ((0, kg), (1, vg)):
            codes, scale = okv4.quantise(x[0, i], gl)
            assert np.array_equal(got[2 * i + 1][:, :rows], scale)
            have = got[2 * i][:, :rows]
            # a zero may carry a sign: compare the values of finite groups
            a, b = okv4.values(have, scale, gl), okv4.values(okv4.pack(codes), scale, gl)
            assert np.array_equal(a, b, equal_nan=True)
        dst = torch.empty((1, 2, 1, rows, 128), dtype=torch.bfloat16, device=dev)
        g.kv4_read_rows([layer], 0, rows, dst)
        assert np.array_equal(dst[0, 1].isnan().cpu().numpy(), np.isnan(okv4.values(got[2][:, :rows], got[3][:, :rows], vg)))


def test_no_room_sets_status_2_and_writes_nothing(dev):
    import tree_verified_block_gb300 as g
    g.reset_device_status()
    gen = W.rng(5)
    host = fresh(gen, 2, 2, 40)
    for T in (25, -1, 2 ** 31 - 1):
        t_len = torch.tensor([T], dtype=torch.int32, device=dev)
        layers = [layer_of(g, h, t_len, dev) for h in host]
        g.kv4_write_rows(bf16_tensor(W.normal_bf16(gen, (2, 2, 2, 16, 128)), dev), layers, 16)
        st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
        g.get_status(st)
        assert st.tolist() == [2, 0, 0, 0, 2, 0]  # reported with walk + commit
        code, _ = g.device_status()
        g.clear_status()
        assert code == 2 and g.device_status()[0] == 0
        for l, h in zip(layers, host):
            assert all(np.array_equal(a, b) for a, b in zip(bytes_of(l), h))


def test_offsets_past_32_bits(dev, clean_status):
    """A cache whose last head starts past 2^32 bytes."""
    import tree_verified_block_gb300 as g
    slots, Hkv, T = 1 << 25, 3, (1 << 25) - 6  # head 2 at 2 * 2^25 * 64 = 2^32 bytes
    t_len = torch.tensor([T], dtype=torch.int32, device=dev)
    layer = g.KV4Layer.empty(Hkv, slots, t_len, device=dev)
    src = W.normal_bf16(W.rng(8), (1, 2, Hkv, 6, 128))
    g.kv4_write_rows(bf16_tensor(src, dev), [layer], 6)
    dst = torch.empty((1, 2, Hkv, 6, 128), dtype=torch.bfloat16, device=dev)
    g.kv4_read_rows([layer], T, 6, dst)
    codes, scale = okv4.quantise(W.bf16_bits_to_f32(src), 1.0)
    assert np.array_equal(dst.double().cpu().numpy(), okv4.values(okv4.pack(codes), scale, 1.0))
    assert int(layer.k[:, :T].count_nonzero()) == 0


def test_another_stream_and_a_graph(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = W.rng(11)
    t_len = torch.tensor([3], dtype=torch.int32, device=dev)
    layers = g.Views([layer_of(g, h, t_len, dev) for h in fresh(gen, 2, 2, 40)])
    src = bf16_tensor(W.normal_bf16(gen, (2, 2, 2, 16, 128)), dev)
    dst = torch.zeros((2, 2, 2, 16, 128), dtype=torch.bfloat16, device=dev)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g.kv4_write_rows(src, layers, 16, stream=side)
    g.kv4_read_rows(layers, 3, 16, dst, stream=side)
    side.synchronize()
    first = dst.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g.kv4_write_rows(src, layers, 16)
        g.kv4_read_rows(layers, 3, 16, dst)
    src.mul_(2)
    dst.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dst, first * 2)  # doubling doubles every scale
