"""Walk + commit on 4-bit caches, and whole rounds on them."""
import numpy as np
import pytest
import torch

import workloads as W
from _kv4_util import attention64, bytes_of, layer_of, random_cache, random_tree, up, upload_tree
from _util import bf16_tensor
from oracle import kv4 as okv4
from oracle import walk as owalk

pytestmark = pytest.mark.gpu


def path_to(t, row):
    path = [row]
    while t["parent"][path[-1]] >= 0:
        path.append(int(t["parent"][path[-1]]))
    return path[::-1]


def argmax_along(gen, t, row):
    a = gen.integers(60000, 90000, len(t["token"])).astype(np.int32)
    p = path_to(t, row)
    for u, v in zip(p, p[1:]):
        a[u] = t["token"][v]
    return a


@pytest.mark.parametrize("B,N,L,n_layers,Hkv,chain", [
    (1, 1, 1, 1, 1, False), (1, 15, 7, 3, 2, False), (1, 16, 16, 36, 8, True), (3, 63, 15, 2, 3, False), (16, 20, 5, 60, 1, False),
    (2, 255, 16, 1, 4, False)])
@pytest.mark.parametrize("gate", [False, True])
def test_commit_moves_the_path_rows(dev, clean_status, B, N, L, n_layers, Hkv, chain, gate):
    import tree_verified_block_gb300 as g
    gen = W.rng(B, N, n_layers)
    rows = N + 1
    trees, args, gaps, hosts, layers, Ts = [], [], [], [], [], []
    t_len = torch.zeros(B, dtype=torch.int32, device=dev)
    for r in range(B):
        T = 5 + 11 * r
        Ts.append(T)
        t_len[r] = T
        t = random_tree(gen, N, L, T, chain)
        trees.append(t)
        args.append(argmax_along(gen, t, [rows - 1, 0, rows // 2][r % 3]))
        gaps.append(gen.random(rows).astype(np.float32))
        n = T + rows + 3 + (T + rows + 3) % 2
        for _ in range(n_layers):
            hosts.append([gen.integers(0, 256, (Hkv, n, w)).astype(np.uint8) for w in (64, 8, 64, 8)])
            layers.append(layer_of(g, hosts[-1], t_len[r:r + 1], dev, t_cap=n - 1 if Hkv > 1 else None))
    i32 = lambda *s: torch.full(s, -7, dtype=torch.int32, device=dev)
    n_acc, tok, root, gated = i32(B), i32(B, L), i32(B), i32(B)
    ws = g.workspace(g.kv4_accept_commit_workspace_bytes(B, n_layers), dev)
    kw = dict(gap=up(np.stack(gaps), dev), gate_threshold=0.1, gated=gated) if gate else {}
    g.kv4_accept_commit([upload_tree(g, t, L, dev) for t in trees], up(np.stack(args), dev), g.Views(layers), n_acc, tok,
                        root, ws, **kw)
    assert int(ws.view(torch.int32).abs().sum()) == 0  # the counters are back at zero
    for r in range(B):
        if gate:
            a, path, acc, nr, gt = owalk.walk_gated(trees[r], args[r], gaps[r], L, np.float32(0.1))
            assert int(gated[r]) == int(gt)
        else:
            a, path, acc, nr = owalk.walk(trees[r], args[r], L)
        T = Ts[r]
        assert int(n_acc[r]) == a and int(root[r]) == nr and int(t_len[r]) == T + a + 1
        assert tok[r, :a].tolist() == acc and tok[r, a:].tolist() == [-7] * (L - a)
        for l in range(n_layers):
            for got, h in zip(bytes_of(layers[r * n_layers + l]), hosts[r * n_layers + l]):
                want = h[:, :got.shape[1]].copy()
                want[:, T:T + a + 1] = h[:, [T + p for p in path]]
                assert np.array_equal(got, want), (r, l)


def test_no_room_sets_status_2_and_moves_nothing(dev):
    import tree_verified_block_gb300 as g
    g.reset_device_status()
    gen = W.rng(5)
    t = random_tree(gen, 15, 7)
    cache = random_cache(gen, 2, 40, 1.0, 1.0)
    t_len = torch.tensor([25], dtype=torch.int32, device=dev)
    layer = layer_of(g, cache, t_len, dev)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    g.kv4_accept_commit(upload_tree(g, t, 7, dev), up(argmax_along(gen, t, 15), dev), layer, z(1), z(7), z(1),
                        g.workspace(256, dev))
    st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
    g.get_status(st)
    assert st.tolist() == [2, 0, 0, 0, 2, 0]
    g.reset_device_status()
    assert int(t_len) == 25 and all(np.array_equal(a, b) for a, b in zip(bytes_of(layer), cache))


def test_rounds_leave_the_cache_that_decoding_one_by_one_leaves(dev, clean_status):
    """Two layers' caches over several captured rounds: rows written, attention,
    walk + commit. After each round the bytes of slots 0..T-1 are those that
    writing the accepted rows one at a time would leave, and the attention of
    every accepted row is what a one-row call on that shorter cache gives."""
    import tree_verified_block_gb300 as g
    gen = W.rng(23)
    n_layers, Hkv, Hq, N, L, cap = 2, 2, 8, 24, 6, 400
    rows = N + 1
    t_len, t_one = (torch.tensor([50], dtype=torch.int32, device=dev) for _ in range(2))
    start = [random_cache(gen, Hkv, cap, 1.0, 0.5) for _ in range(n_layers)]
    layers = g.Views([layer_of(g, c, t_len, dev, 1.0, 0.5) for c in start])
    ones = g.Views([layer_of(g, c, t_one, dev, 1.0, 0.5) for c in start])
    tree = g.Tree(N, L, dev)
    trees = g.Views([tree])
    views = [g.Views([l]) for l in layers]
    one_views = [g.Views([l]) for l in ones]
    src = torch.zeros(n_layers, 2, Hkv, rows, 128, dtype=torch.bfloat16, device=dev)
    q = torch.zeros(n_layers, 1, rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    out = torch.zeros_like(q)
    argmax = torch.zeros(1, rows, dtype=torch.int32, device=dev)
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    n_acc, tok, root = z(1), z(1, L), z(1)
    ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, views[0]), dev)
    wsc = g.workspace(g.kv4_accept_commit_workspace_bytes(1, n_layers), dev)

    def round_():
        g.kv4_write_rows(src, layers, rows)
        for l in range(n_layers):
            g.kv4_tree_attention(q[l], views[l], trees, 0.09, out[l], ws)
        g.kv4_accept_commit(trees, argmax, layers, n_acc, tok, root, wsc)

    round_()  # first calls outside the capture
    t_len.fill_(50)
    for l, c in zip(layers, start):
        for dst, a in zip((l.k, l.k_scale, l.v, l.v_scale), c):
            dst.copy_(up(a, dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        round_()
    T = 50
    ws1 = g.workspace(g.kv4_tree_attention_workspace_bytes(1, Hq, one_views[0]), dev)
    for step in range(5):
        t = random_tree(gen, N, L, T)
        new = upload_tree(g, t, L, dev)
        for name in ("token", "parent", "depth", "pos_id", "anc"):
            getattr(tree, name).copy_(getattr(new, name))
        a_host = argmax_along(gen, t, int(gen.integers(0, rows)))
        argmax.copy_(up(a_host, dev)[None])
        src.copy_(bf16_tensor(W.normal_bf16(gen, tuple(src.shape)), dev))
        q.copy_(bf16_tensor(W.normal_bf16(gen, tuple(q.shape)), dev))
        graph.replay()
        a, path, acc, nr = owalk.walk(t, a_host, L)
        assert int(n_acc) == a and int(root) == nr and tok[0, :a].tolist() == acc
        for p in path:
            g.kv4_write_rows(src[:, :, :, p:p + 1].contiguous(), ones, 1)
            for l in range(n_layers):
                o1 = torch.zeros(1, 1, Hq, 128, dtype=torch.bfloat16, device=dev)
                g.kv4_tree_attention(q[l, :, p:p + 1].contiguous(), one_views[l], None, 0.09, o1, ws1)
                o, tol = attention64(q[l, 0, p:p + 1], bytes_of(ones[l]), T, np.ones((1, 1), bool), 0.09, 1.0, 0.5, dev)
                assert torch.all((o1[0].double() - o).abs() <= tol)
                assert torch.all((out[l, 0, p:p + 1].double() - o).abs() <= tol)
            t_one += 1
            T += 1
        assert int(t_len) == T == int(t_one)
        for l in range(n_layers):
            for x, y in zip(bytes_of(layers[l]), bytes_of(ones[l])):
                assert np.array_equal(x[:, :T], y[:, :T])


def test_a_layer_from_projection_to_output_on_a_4_bit_cache(dev, clean_status):
    """qk_norm_rope of the projected rows into bf16 rows, those into the 4-bit
    cache, attention over it: against the formulas on what each step stores."""
    import tree_verified_block_gb300 as g
    from oracle import rope as orope
    gen = W.rng(29)
    Hq, Hkv, T, N = 8, 2, 333, 40
    rows = N + 1
    t = random_tree(gen, N, 8, T)
    cache = random_cache(gen, Hkv, 400, 1.0, 1.0)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
    qkv = bf16_tensor(W.normal_bf16(gen, (rows, (Hq + 2 * Hkv) * 128)), dev)
    w = torch.from_numpy(gen.uniform(0.5, 1.5, 128).astype(np.float32)).to(dev)
    # a time, height and width position for every row, as an image's tokens have
    pos = np.stack([t["pos_id"], t["pos_id"] % 17, t["pos_id"] % 23]).astype(np.int32)
    staged = torch.zeros(1, 2, Hkv, rows, 128, dtype=torch.bfloat16, device=dev)
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    q = torch.empty(1, rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    out = torch.empty_like(q)
    sec = [24, 20, 20]
    g.qk_norm_rope(qkv, Hq, w, w, 1e-6, up(pos, dev), g.Rope(128, 1e6, sec, True), q, g.KVLayer(staged[0, 0], staged[0, 1], zero))
    g.kv4_write_rows(staged, [layer], rows)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, t, 8, dev)], 128 ** -0.5, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, [layer]), dev))
    x = qkv.double().cpu().numpy().reshape(rows, -1, 128)
    wk = w.double().cpu().numpy()
    for got, want in ((q[0], orope.qk_norm_rope(x[:, :Hq], wk, pos, 1e6, sec, True)),
                      (staged[0, 0].transpose(0, 1), orope.qk_norm_rope(x[:, Hq:Hq + Hkv], wk, pos, 1e6, sec, True))):
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17)
    rows16 = W.bf16_bits_to_f32(staged.view(torch.int16).cpu().numpy().view(np.uint16))
    for i in (0, 1):
        codes, scale = okv4.quantise(rows16[0, i], 1.0)
        cache[2 * i][:, T:T + rows], cache[2 * i + 1][:, T:T + rows] = okv4.pack(codes), scale
    for a, b in zip(bytes_of(layer), cache):
        assert np.array_equal(a, b)
    o, tol = attention64(q[0], cache, T, t["seen"], 128 ** -0.5, 1.0, 1.0, dev)
    assert torch.all((out[0].double() - o).abs() <= tol)
