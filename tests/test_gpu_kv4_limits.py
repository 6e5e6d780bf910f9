"""Attention over 4-bit caches at the limits of its formats: scales that are not
numbers next to the end of the prefix, weights far below the largest, query rows
that are not finite."""
import math

import numpy as np
import pytest
import torch

import workloads as W
from _kv4_tight import tight64
from _kv4_util import anc_words, layer_of, random_cache, random_tree, up, upload_tree
from _util import bf16_tensor
from oracle import kv4 as okv4

pytestmark = pytest.mark.gpu


# Lengths whose last prefix tiles are cut by the end of a block's part: equal
# parts of 5, 6, 7, ... units of 32 slots, and runs over the list of all groups.
@pytest.mark.parametrize("N,Hq,Hkv,Ts", [
    (63, 32, 8, [2800]), (63, 32, 8, [3097]), (63, 32, 8, [3615]), (63, 8, 8, [2431]), (19, 64, 8, [2579]), (255, 32, 8, [322]),
    (255, 32, 8, [396]), (255, 32, 8, [1728]), (63, 32, 8, [512, 762, 1133, 1686, 2508, 3730, 5548, 8192]),
    (63, 32, 8, [1191, 3539, 612, 713, 148, 1640, 1798, 546]), (0, 32, 8, [2800]), (0, 8, 8, [3097, 700]), (3, 32, 8, [2431])])
def test_a_scale_that_is_no_number_at_the_end_of_the_prefix_reaches_every_row(dev, clean_status, N, Hq, Hkv, Ts):
    import tree_verified_block_gb300 as g
    gen = W.rng(83, N, Hq)
    B, rows, G = len(Ts), N + 1, Hq // Hkv
    layers, trees = [], []
    for T in Ts:
        layers.append(layer_of(g, random_cache(gen, Hkv, T + rows + (T + rows) % 2, 1.0, 1.0),
                               torch.tensor([T], dtype=torch.int32, device=dev), dev))
        trees.append(upload_tree(g, random_tree(gen, N, 16, T), 16, dev))
    views, c_trees = g.Views(layers), g.Views(trees)
    q = bf16_tensor(W.normal_bf16(gen, (B, rows, Hq, 128)), dev)
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, views), dev)
    out = torch.zeros_like(q)
    head = torch.arange(Hkv, device=dev)
    for name in ("v_scale", "k_scale"):
        for first in range(128 // Hkv):
            was = []
            for layer, T in zip(layers, Ts):  # another of the last 128 prefix slots in every kv head
                scales, slot = getattr(layer, name), T - 128 + first * Hkv + head
                was.append((scales, slot, scales[head, slot, 3].clone()))
                scales[head, slot, 3] = 0x7F
            g.kv4_tree_attention(q, views, c_trees, 0.09, out, ws)
            gone = out.isnan().any(-1).view(B, rows, Hkv, G)
            assert gone.all(), (name, first, (~gone).nonzero()[0].tolist())
            for scales, slot, old in was:
                scales[head, slot, 3] = old
        g.kv4_tree_attention(q, views, c_trees, 0.09, out, ws)
        assert not out.isnan().any()


def sinks(Hkv, n, T):
    """Bytes of a cache of n slots: every 96th prefix slot has a large K in its
    first dim and V = 0, the others K = 0 and V that differs by dim only, at the
    largest scale."""
    code = np.zeros((Hkv, n, 128), np.uint8)
    at = np.arange(5, T, 96)
    k = code.copy()
    k[:, at, 0] = 7  # magnitude 6
    v = code.copy()
    v[:] = np.resize(np.array([1, 7, 10, 15, 4, 13], np.uint8), 128)
    v[:, at] = 0
    one = np.full((Hkv, n, 8), 0x38, np.uint8)
    return [okv4.pack(k), one, okv4.pack(v), np.full_like(one, 0x7E)]


@pytest.mark.parametrize("below", [20.7, 25.5])
@pytest.mark.parametrize("N,Hq,Hkv,T", [(0, 1, 1, 20000), (0, 32, 8, 5000), (9, 1, 1, 20000), (3, 8, 2, 3001), (40, 1, 1, 20000),
                                        (63, 8, 1, 20000), (63, 32, 8, 4096), (255, 2, 1, 9001)])
def test_many_small_weights_beside_large_ones_are_kept(dev, clean_status, N, Hq, Hkv, T, below):
    """Attention sinks: slots of a large weight and V = 0 beside many of 2^-below
    of it, which make up the whole output."""
    import tree_verified_block_gb300 as g
    gen = W.rng(89, N)
    rows = N + 1
    cache = sinks(Hkv, T + rows + (T + rows) % 2, T)
    t = random_tree(gen, N, 16, T)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
    q = torch.zeros(1, rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    q[..., 0] = 1
    scale = below * math.log(2) / 6
    out = torch.zeros_like(q)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], scale, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    o, tol = tight64(q[0], cache, T, t["seen"], scale, 1.0, 1.0, dev)
    assert torch.all(tol < 0.04 * o.abs())  # of use: the tolerance is far below the output
    err = (out[0].double() - o).abs()
    assert torch.all(err <= tol), float((err / tol).max())


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 4, 2), (3, 8, 2), (9, 2, 2), (40, 8, 2)])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), float("-inf")])
def test_a_query_row_that_sees_nothing_is_zero_whatever_it_holds(dev, clean_status, N, Hq, Hkv, what):
    import tree_verified_block_gb300 as g
    gen = W.rng(97, N)
    rows = N + 1
    seen = np.eye(rows, dtype=bool)
    seen[0] = seen[N] = False
    t = random_tree(gen, N, 16)
    t["anc"] = anc_words(seen)
    layer = layer_of(g, random_cache(gen, Hkv, rows + rows % 2, 1.0, 1.0), torch.zeros(1, dtype=torch.int32, device=dev), dev)
    q = bf16_tensor(W.normal_bf16(gen, (1, rows, Hq, 128)), dev)
    q[0, 0, :, 7] = what
    q[0, N, Hq - 1] = what
    out = torch.full_like(q, 3.0)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], 0.09, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    assert torch.all(out[0, 0] == 0) and torch.all(out[0, N] == 0)
    assert not out.isnan().any()


@pytest.mark.parametrize("N,Hq,Hkv,T", [(0, 8, 2, 300), (0, 4, 4, 5000), (3, 8, 2, 300), (9, 2, 2, 3000), (40, 8, 2, 300), (63, 32, 8, 4000),
                                        (100, 8, 1, 2000)])
@pytest.mark.parametrize("size", range(20, 68, 2))
def test_scores_of_any_size_leave_the_largest_one_s_value(dev, clean_status, N, Hq, Hkv, T, size):
    """Scores of about 2^size (log2), far past the fp32 numbers that are whole:
    the largest one's V row is the output where no other is near it.

    Near: the fp32 scores are off by 132 steps of 2^-23 of sum |q| |k|, as in
    tight64, each; twice that, and 40 more for the others' weights."""
    import tree_verified_block_gb300 as g
    gen = W.rng(109, N, size)
    rows = N + 1
    cache = random_cache(gen, Hkv, T + rows + (T + rows) % 2, 1.0, 1.0)
    t = random_tree(gen, N, 16, T)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
    q = bf16_tensor(W.normal_bf16(gen, (1, rows, Hq, 128)), dev)
    scale = 2.0 ** size / 40
    out = torch.zeros_like(q)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], scale, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    n, G = T + rows, Hq // Hkv
    k = up(okv4.values(cache[0][:, :n], cache[1][:, :n], 1.0), dev)
    v = up(okv4.values(cache[2][:, :n], cache[3][:, :n], 1.0), dev)
    vis = torch.cat((torch.ones(rows, T, dtype=torch.bool), torch.from_numpy(t["seen"])), 1).to(dev)
    clear = 0
    for h in range(Hq):
        x = q[0, :, h].double()
        s = (x @ k[h // G].t()).masked_fill(~vis, -torch.inf)
        top, at = s.topk(2, -1)
        off = (x.abs() @ k[h // G].abs().t()).amax(-1) * 132 * 2 ** -23
        one = top[:, 0] - top[:, 1] > 2 * off + 40 / scale
        o = v[h // G][at[:, 0]]
        assert not out[0, :, h].isnan().any()
        assert torch.all(((out[0, :, h].double() - o).abs() <= (2 ** -8 + 2 ** -10) * o.abs() + 2 ** -25)[one])
        clear += int(one.sum())
    assert clear >= rows * Hq // 2


@pytest.mark.parametrize("N,Hq,Hkv", [(0, 1, 1), (9, 1, 1), (40, 1, 1), (255, 1, 1)])
@pytest.mark.parametrize("run", [64, 256])
def test_climbing_scores_of_any_size_give_a_mean_of_the_values(dev, clean_status, N, Hq, Hkv, run):
    """Scores that climb by up to 8 (log2) every 64 slots or every 256, the most
    for which sums need not be rescaled, on top of 2^20 to 2^30: whatever fp32
    makes of them, the output is a mean of V rows, which are 1 to 6 here."""
    import tree_verified_block_gb300 as g
    gen = W.rng(113, N)
    rows, T = N + 1, 64 * run
    n = T + rows + (T + rows) % 2
    k = np.zeros((Hkv, n, 128), np.uint8)
    k[..., 0] = 7
    step = np.minimum(np.arange(n) // run, 63)
    for bit in range(6):
        k[..., 16 + bit] = 2 * (step >> bit & 1)  # 1 or 0
    ks = np.full((Hkv, n, 8), 0x38, np.uint8)
    ks[..., 0] = 0x7E  # 6 * 448
    v = gen.integers(2, 8, (Hkv, n, 128), dtype=np.uint8)
    cache = [okv4.pack(k), ks, okv4.pack(v), np.full((Hkv, n, 8), 0x38, np.uint8)]
    t = random_tree(gen, N, 16, T)
    layer, tree = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev), upload_tree(g, t, 16, dev)
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev)
    out = torch.zeros(1, rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    for base in np.arange(20, 31, 0.25):
        for climb in (7.5, 7.875, 7.9375, 8.0):
            for sign in (1, -1):
                q = torch.zeros_like(out)
                q[..., 0] = sign * 2.0 ** base / 2688
                q[..., 16:22] = torch.tensor([climb * 2.0 ** b for b in range(6)], dtype=torch.bfloat16)
                g.kv4_tree_attention(q, layer, tree, math.log(2), out, ws)
                assert torch.all((out >= 1) & (out <= 6)), (base, climb, sign)
