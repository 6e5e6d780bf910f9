"""Tree attention over 4-bit caches against the formula in 64 bits on the
values that the bytes stand for."""
import numpy as np
import pytest
import torch

import workloads as W
from _kv4_util import attention64, layer_of, random_cache, random_tree, up, upload_tree
from _util import bf16_tensor

pytestmark = pytest.mark.gpu

KG, VG = 0.75, 5.5 / 2688


def check(dev, Ts, N, Hq, Hkv, seed=0, seen=None, gap=0, spare=0, q_std=1.0, trees_null=False, kv_std=1.0, kg=KG, vg=VG):
    import tree_verified_block_gb300 as g
    B, rows, L = len(Ts), N + 1, 16
    gen = W.rng(seed, N, B, Hq)
    caches, layers, trees, seens = [], [], [], []
    for T in Ts:
        n = T + rows + spare
        c = random_cache(gen, Hkv, n + n % 2 + gap, kg, vg, kv_std)
        for a in c:  # slots past the tree: anything, NaN scales among it
            a[:, T + rows:] = 255
        t = random_tree(gen, N, L, T)
        if seen is not None:
            from _kv4_util import anc_words
            t["seen"] = seen
            t["anc"] = anc_words(seen)
        caches.append(c)
        layers.append(layer_of(g, c, torch.tensor([T], dtype=torch.int32, device=dev), dev, kg, vg, n + n % 2 if gap else None))
        trees.append(upload_tree(g, t, L, dev))
        seens.append(t["seen"])
    q = bf16_tensor(W.normal_bf16(gen, (B, rows, Hq, 128), q_std), dev)
    out = torch.full_like(q, 3.0)
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, layers), dev)
    views = g.Views(layers)
    g.kv4_tree_attention(q, views, None if trees_null else trees, 128 ** -0.5, out, ws)
    again = torch.full_like(q, -3.0)
    g.kv4_tree_attention(q, views, None if trees_null else trees, 128 ** -0.5, again, ws)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))  # the same bits every time
    for r, T in enumerate(Ts):
        o, tol = attention64(q[r], caches[r], T, seens[r], 128 ** -0.5, kg, vg, dev)
        err = (out[r].double() - o).abs()
        assert torch.all(err <= tol), (r, T, float((err / tol).max()))
    return out


# one row (decoding), with every group size, from an empty prefix to ranges that split over many blocks
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (4, 2), (8, 2), (32, 8), (16, 2)])
@pytest.mark.parametrize("T", [0, 1, 31, 32, 100, 127, 1000, 5000])
def test_one_row(dev, clean_status, T, Hq, Hkv):
    check(dev, [T], 0, Hq, Hkv, spare=7)


@pytest.mark.parametrize("N,Hq,Hkv", [(1, 8, 2), (3, 8, 2), (3, 4, 4), (15, 2, 2), (7, 4, 2), (15, 1, 1), (4, 8, 2), (16, 1, 1),
                                      (8, 4, 2), (31, 8, 2), (63, 8, 2), (62, 4, 1), (64, 4, 4), (100, 8, 1), (127, 2, 1), (255, 4, 2),
                                      (255, 8, 1), (200, 1, 1)])
@pytest.mark.parametrize("T", [0, 3, 255, 1337])
def test_tree_rows(dev, clean_status, N, Hq, Hkv, T):
    check(dev, [T], N, Hq, Hkv)


@pytest.mark.parametrize("N,Hq,Hkv,Ts", [
    (0, 32, 8, [0, 1, 5, 40, 333, 2000, 64, 63, 65, 1, 900, 17, 128, 127, 129, 4000]), (0, 8, 1, [3000, 10]),
    (2, 8, 2, [10, 700, 0]), (15, 8, 2, [100, 1500, 4000]), (63, 8, 2, [100, 1500, 4000]), (63, 32, 8, [512, 700, 1131, 9, 2498]),
    (255, 4, 4, [0, 300])])
def test_ragged_batch(dev, clean_status, N, Hq, Hkv, Ts):
    check(dev, Ts, N, Hq, Hkv, spare=5)


def test_long_prefix(dev, clean_status):
    check(dev, [40001], 0, 4, 1)
    check(dev, [30000], 9, 4, 1)
    check(dev, [20003], 63, 2, 1)


def test_gap_between_heads_and_odd_capacity(dev, clean_status):
    check(dev, [77], 12, 8, 2, gap=6)
    check(dev, [78], 0, 8, 2, gap=30)


def test_no_trees_is_a_row_that_sees_itself(dev, clean_status):
    a = check(dev, [77, 500], 0, 8, 2, trees_null=True)
    b = check(dev, [77, 500], 0, 8, 2)
    assert torch.equal(a, b)


@pytest.mark.parametrize("N,Hq,Hkv", [(9, 2, 2), (3, 8, 2), (40, 8, 2), (130, 2, 1)])
def test_rows_that_see_nothing_are_zero(dev, clean_status, N, Hq, Hkv):
    seen = np.tril(W.rng(3).random((N + 1, N + 1)) < 0.4)
    seen[0] = False
    seen[N] = False
    out = check(dev, [0], N, Hq, Hkv, seen=seen)
    assert torch.all(out[0, 0] == 0) and torch.all(out[0, N] == 0)
    check(dev, [5], N, Hq, Hkv, seen=seen)


@pytest.mark.parametrize("q_std", [1e-30, 1e-6, 40.0, 1e4])
@pytest.mark.parametrize("N", [2, 40])
def test_small_and_large_queries(dev, clean_status, q_std, N):
    """Powers of two move a query into f16's range; large scores leave one key."""
    check(dev, [300], N, 8, 2, q_std=q_std, kv_std=0.5)


@pytest.mark.parametrize("N,Hq,Hkv,T", [(0, 8, 2, 100), (6, 4, 2, 64), (30, 8, 2, 200), (63, 4, 1, 1000)])
def test_not_a_number_reaches_only_the_rows_that_see_it(dev, clean_status, N, Hq, Hkv, T):
    import tree_verified_block_gb300 as g
    gen = W.rng(7, N)
    rows = N + 1
    t = random_tree(gen, N, 16, T)
    q = bf16_tensor(W.normal_bf16(gen, (1, rows, Hq, 128)), dev)
    for which in (1, 3):  # a scale of K, of V
        cache = random_cache(gen, Hkv, T + rows + rows % 2 + T % 2 + 8, 1.0, 1.0)
        bad = rows // 2
        cache[which][0, T + bad, 5] = 0x7F
        layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
        out = torch.zeros_like(q)
        g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], 0.09, out,
                             g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
        hit = torch.zeros(rows, Hq, dtype=torch.bool, device=dev)
        hit[up(t["seen"][:, bad], dev), :Hq // Hkv] = True
        assert torch.equal(out[0].isnan().any(-1), hit)
        o, tol = attention64(q[0], cache, T, t["seen"], 0.09, 1.0, 1.0, dev)
        fine = ~hit
        assert torch.all((out[0].double() - o).abs()[fine] <= tol[fine])
        # the same in the prefix reaches every row of the kv head
        if T > 10:
            cache[which][0, T + bad, 5] = 0x38
            cache[which][Hkv - 1, 7, 2] = 0x7F
            layer = layer_of(g, cache, layer.t_len, dev)
            g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 16, dev)], 0.09, out,
                                 g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
            assert out[0, :, -1].isnan().any(-1).all() and not out[0, :, :Hq - Hq // Hkv].isnan().any()


def test_not_finite_queries_stay_in_their_row(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = W.rng(9)
    for N, T in ((0, 40), (3, 40), (50, 300)):
        rows = N + 1
        q = bf16_tensor(W.normal_bf16(gen, (1, rows, 8, 128)), dev)
        q[0, 0, 1, 3] = float("nan")
        q[0, N, 6, 100] = float("-inf")
        cache = random_cache(gen, 2, T + rows + 9 + (T + rows + 9) % 2, 1.0, 1.0)
        layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
        out = torch.zeros_like(q)
        g.kv4_tree_attention(q, [layer], [upload_tree(g, random_tree(gen, N, 16, T), 16, dev)], 0.09, out,
                             g.workspace(g.kv4_tree_attention_workspace_bytes(rows, 8, [layer]), dev))
        hit = torch.zeros(rows, 8, dtype=torch.bool, device=dev)
        hit[0, 1] = hit[N, 6] = True
        assert torch.equal(out[0].isnan().any(-1), hit)


@pytest.mark.parametrize("N", [0, 20])
def test_no_room_sets_status_2_and_leaves_out(dev, N):
    import tree_verified_block_gb300 as g
    g.reset_device_status()
    gen = W.rng(5)
    cap = 64 + 2 * N
    cache = random_cache(gen, 2, cap, 1.0, 1.0)
    ts = [torch.tensor([t], dtype=torch.int32, device=dev) for t in (cap - N, 10)]
    layers = [layer_of(g, cache, t, dev) for t in ts]
    t = random_tree(gen, N, 16)
    q = bf16_tensor(W.normal_bf16(gen, (2, N + 1, 4, 128)), dev)
    out = torch.full_like(q, 7.0)
    g.kv4_tree_attention(q, layers, [upload_tree(g, t, 16, dev)] * 2, 0.1, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(N + 1, 4, layers), dev))
    st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
    g.get_status(st)
    assert st.tolist() == [2, 0, 2, 0, 0, 0]
    g.reset_device_status()
    assert torch.all(out[0] == 7)
    o, tol = attention64(q[1], cache, 10, t["seen"], 0.1, 1.0, 1.0, dev)
    assert torch.all((out[1].double() - o).abs() <= tol)


@pytest.mark.parametrize("N", [0, 10, 63])
def test_graph_with_a_growing_prefix_and_a_shared_workspace(dev, clean_status, N):
    """T is read on the device: one captured call serves every length; two
    graphs replayed in turn may share the workspace."""
    import tree_verified_block_gb300 as g
    gen = W.rng(13, N)
    rows, cap = N + 1, 3000
    cache = random_cache(gen, 2, cap, 1.0, 1.0)
    t_len = torch.zeros(1, dtype=torch.int32, device=dev)
    layer = g.Views([layer_of(g, cache, t_len, dev)])
    t = random_tree(gen, N, 16)
    tree = g.Views([upload_tree(g, t, 16, dev)])
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, 8, layer), dev)
    qs = [bf16_tensor(W.normal_bf16(gen, (1, rows, 8, 128)), dev) for _ in range(2)]
    outs = [torch.zeros_like(q) for q in qs]
    g.kv4_tree_attention(qs[0], layer, tree, 0.09, outs[0], ws)
    graphs = []
    for q, out in zip(qs, outs):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            g.kv4_tree_attention(q, layer, tree, 0.09, out, ws)
        graphs.append(graph)
    for T in (0, 5, 130, 2000, cap - rows):
        t_len.fill_(T)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        torch.cuda.synchronize()
        for q, out in zip(qs, outs):
            o, tol = attention64(q[0], cache, T, t["seen"], 0.09, 1.0, 1.0, dev)
            assert torch.all((out[0].double() - o).abs() <= tol), T


def test_two_calls_at_once_on_two_streams(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = W.rng(17)
    for N in (0, 30):
        rows, T = N + 1, 1500
        cache = random_cache(gen, 2, T + rows + 1 + (T + rows + 1) % 2, 1.0, 1.0)
        layer = g.Views([layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)])
        t = random_tree(gen, N, 16)
        tree = g.Views([upload_tree(g, t, 16, dev)])
        work = []
        for _ in range(2):
            q = bf16_tensor(W.normal_bf16(gen, (1, rows, 8, 128)), dev)
            work.append((q, torch.zeros_like(q), g.workspace(g.kv4_tree_attention_workspace_bytes(rows, 8, layer), dev),
                         torch.cuda.Stream()))
        torch.cuda.synchronize()
        for _ in range(10):
            for q, out, ws, s in work:
                g.kv4_tree_attention(q, layer, tree, 0.09, out, ws, stream=s)
        torch.cuda.synchronize()
        for q, out, _, _ in work:
            o, tol = attention64(q[0], cache, T, t["seen"], 0.09, 1.0, 1.0, dev)
            assert torch.all((out[0].double() - o).abs() <= tol)
