"""Attention over 4-bit caches at the limits of its formats: scales that are not
numbers next to the end of the prefix, weights far below the largest, query rows
that are not finite."""
import numpy as np
import pytest
import torch

import workloads as W
from _kv4_util import layer_of, random_cache, random_tree, upload_tree
from _util import bf16_tensor

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
