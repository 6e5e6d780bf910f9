"""Attention over long 4-bit caches, where one slot's share of an ordinary output
is below its rounding: every slot is asked for by a query that only its key
answers, and summed once with the others under equal weights."""
import numpy as np
import pytest
import torch

import workloads as W
from _kv4_tight import tight64
from _kv4_util import layer_of, random_cache, random_tree, up, upload_tree
from _util import bf16_tensor
from oracle import kv4 as okv4

pytestmark = pytest.mark.gpu

# up to 8 and 16 query rows per kv head, more (one, two and three tiles of 128, a
# pair and one over), several heads
CASES = [(0, 8, 1, 131072), (1, 8, 1, 131072), (63, 8, 1, 131072), (39, 1, 1, 40001), (255, 1, 1, 20003), (47, 8, 1, 40001),
         (63, 8, 2, 30011), (0, 8, 2, 30011)]


@pytest.mark.parametrize("N,Hq,Hkv,T", CASES)
def test_every_slot_is_found_by_its_key(dev, clean_status, N, Hq, Hkv, T):
    """K rows of random signs: q = the K row of a slot scores 128 there and, over
    all pairs here, below 90 elsewhere (8 standard deviations of 128 signs), so
    the others' weights are under 2^(-38 * 0.9 / ln 2) = 2^-49 of it, 131072 of
    them with |v| <= 6 under 2^-29, and the output is the slot's V row: a code,
    which bf16 holds and the weights' roundings (2^-11) do not move, or 2^-29
    where that is 0."""
    import tree_verified_block_gb300 as g
    gen = W.rng(101, N, Hkv)
    rows, G = N + 1, Hq // Hkv
    n = T + rows + (T + rows) % 2
    one = np.full((Hkv, n, 8), 0x38, np.uint8)
    k = np.where(gen.random((Hkv, n, 128)) < 0.5, 2, 10).astype(np.uint8)  # 1 and -1
    v = gen.integers(0, 16, (Hkv, n, 128), dtype=np.uint8)
    v[v == 8] = 0
    layer = g.Views([layer_of(g, [okv4.pack(k), one, okv4.pack(v), one], torch.tensor([T], dtype=torch.int32, device=dev), dev)])
    tree = g.Views([upload_tree(g, random_tree(gen, N, 16, T), 16, dev)])
    magnitude = torch.tensor([*okv4.MAGNITUDES, *-okv4.MAGNITUDES], dtype=torch.bfloat16, device=dev)
    ks, vs = magnitude[up(k, dev).int()], magnitude[up(v, dev).int()]
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, layer), dev)
    head = torch.arange(Hkv, device=dev)[:, None]
    for first in range(0, T, rows * G):
        slot = (first + torch.arange(rows * G, device=dev)).clamp(max=T - 1).expand(Hkv, -1)
        q = ks[head, slot].view(Hkv, rows, G, 128).transpose(0, 1).reshape(1, rows, Hq, 128)
        want = vs[head, slot].view(Hkv, rows, G, 128).transpose(0, 1).reshape(1, rows, Hq, 128)
        out = torch.full_like(q, 9.0)
        g.kv4_tree_attention(q, layer, tree, 0.9, out, ws)
        off = (out - want).abs() > 2 ** -29
        assert not off.any(), (first, off.any(-1).nonzero()[0].tolist())


@pytest.mark.parametrize("N,Hq,Hkv,T", CASES)
def test_every_slot_counts_once(dev, clean_status, N, Hq, Hkv, T):
    """q = 0: all weights are the same number, and V has +1 or -1 by the bits of
    the slot's index (dim d: bit d mod 18), so the sums nearly cancel and a slot,
    a unit of 32 or a tile that is left out, taken twice or taken for another
    shows in the dim of one of its bits.

    Tolerance: the output's rounding, and the weights' (2^-11, the same for every
    slot), 2^-8 + 2^-11 of |o|; a part's O / l rounded to f16, 2^-11 of |O_p| / l:
    consecutive slots' bits b sum to at most 2^b, over at most as many parts as
    there are SMs; 2^-20 for the fp32 factors of the parts (the sums are whole
    numbers of weights, exact)."""
    import tree_verified_block_gb300 as g
    gen = W.rng(103, N, Hkv)
    rows = N + 1
    n = T + rows + (T + rows) % 2
    bit = np.arange(128) % 18
    v = np.broadcast_to(np.where(np.arange(n)[:, None] >> bit & 1, 10, 2).astype(np.uint8), (Hkv, n, 128))
    cache = random_cache(gen, Hkv, n, 1.0, 1.0)
    cache[2], cache[3] = okv4.pack(v), np.full((Hkv, n, 8), 0x38, np.uint8)
    t = random_tree(gen, N, 16, T)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
    q = torch.zeros(1, rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    out = torch.full_like(q, 9.0)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], 0.9, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    sign = up(np.where(np.arange(n)[:, None] >> bit & 1, -1.0, 1.0), dev)
    seen = up(t["seen"].astype(np.float64), dev)
    count = T + seen.sum(1, keepdim=True)
    o = (sign[:T].sum(0) + seen @ sign[T:T + rows]) / count
    sms = torch.cuda.get_device_properties(dev).multi_processor_count
    part = up(np.minimum(1.0, sms * 2.0 ** bit / T), dev)
    tol = (2 ** -8 + 2 ** -11) * o.abs() + 2 ** -11 * part + 2 ** -20
    err = (out[0].double() - o[:, None]).abs()
    assert torch.all(err <= tol[:, None]), float((err / tol[:, None]).max())
    # the tolerance shows a slot, a unit and a tile that are left out of the reference
    for size in (1, 32, 128):
        share = sign[:T // size * size].view(-1, size, 128).sum(1).abs() / T
        assert torch.all((share > 2.5 * tol.amax(0)).any(1)), size


@pytest.mark.parametrize("N,Hq,Hkv,T", [(0, 8, 1, 131072), (1, 8, 1, 131072), (63, 2, 1, 131072), (63, 8, 2, 40001), (0, 32, 8, 9999)])
@pytest.mark.parametrize("q_std", [1.0, 4.0])
def test_long_random_rows(dev, clean_status, N, Hq, Hkv, T, q_std):
    import tree_verified_block_gb300 as g
    gen = W.rng(107, N, Hkv)
    rows, kg, vg = N + 1, 0.75, 5.5 / 2688
    cache = random_cache(gen, Hkv, T + rows + (T + rows) % 2, kg, vg)
    t = random_tree(gen, N, 16, T)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev, kg, vg)
    q = bf16_tensor(W.normal_bf16(gen, (1, rows, Hq, 128), q_std), dev)
    out = torch.full_like(q, 9.0)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], 128 ** -0.5, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    o, tol = tight64(q[0], cache, T, t["seen"], 128 ** -0.5, kg, vg, dev)
    err = (out[0].double() - o).abs()
    assert torch.all(err <= tol), float((err / tol).max())
