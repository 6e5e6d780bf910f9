"""The 4-bit cache and norm + rotary calls next to each other and to the calls
on 16-bit caches: one workspace for calls of every shape, more groups than
blocks, rows that the next call reads as its prefix, the bounds-checked build."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import workloads as W
from _kv4_util import anc_words, attention64, layer_of, random_cache, random_tree, up, upload_tree
from _util import bf16_tensor
from test_gpu_kv4_attention import check

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_DIR = os.path.join(os.path.dirname(HERE), "tree_verified_block_gb300", "_lib")


def test_one_workspace_serves_calls_of_every_shape(dev, clean_status):
    """Decoding, trees of few and of many query rows and walk + commit in turn on
    one workspace, zero-filled once: each gives what it gives on its own."""
    import tree_verified_block_gb300 as g
    gen = W.rng(41)
    calls = []
    for N, Hq, Hkv, Ts in ((0, 8, 8, [5000, 700, 40, 3000]), (63, 8, 2, [900, 2000]), (3, 8, 2, [6000]), (15, 16, 16, [300, 1200]),
                           (0, 4, 1, [20000]), (100, 8, 1, [2500]), (0, 32, 8, [100] * 16)):
        rows = N + 1
        layers, trees = [], []
        for T in Ts:
            n = T + rows
            layers.append(layer_of(g, random_cache(gen, Hkv, n + n % 2, 1.0, 0.5), torch.tensor([T], dtype=torch.int32, device=dev),
                                   dev, 1.0, 0.5))
            trees.append(upload_tree(g, random_tree(gen, N, 8, T), 8, dev))
        q = bf16_tensor(W.normal_bf16(gen, (len(Ts), rows, Hq, 128)), dev)
        calls.append((q, g.Views(layers), g.Views(trees), g.kv4_tree_attention_workspace_bytes(rows, Hq, layers)))
    ws = g.workspace(max(c[3] for c in calls), dev)
    want = []
    for q, layers, trees, size in calls:
        want.append(torch.zeros_like(q))
        g.kv4_tree_attention(q, layers, trees, 0.09, want[-1], g.workspace(size, dev))
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    for _ in range(3):
        for (q, layers, trees, _), o in zip(calls, want):
            out = torch.zeros_like(q)
            g.kv4_tree_attention(q, layers, trees, 0.09, out, ws)
            assert torch.equal(out.view(torch.int16), o.view(torch.int16))
            if trees[0].N and len(trees) > 1:  # nothing matches: T moves by one, and back
                B, rows = len(trees), trees[0].rows
                g.kv4_accept_commit(trees, torch.full((B, rows), -5, dtype=torch.int32, device=dev), layers, z(B), z(B, 8), z(B), ws)
                for l in layers:
                    l.t_len -= 1


# more groups (request, kv head, pair of query tiles) than blocks, an odd number
# of query tiles per kv head, and blocks with pairs of query tiles and single ones
# in every order
@pytest.mark.parametrize("N,Hq,Hkv,Ts", [
    (0, 32, 32, [300 + 37 * r for r in range(16)]), (0, 320, 320, [40, 90]), (3, 64, 32, [5, 0, 77, 1000] * 4),
    (20, 16, 16, [64, 200, 30, 7] * 4), (130, 16, 8, [300, 20, 700]), (100, 200, 200, [150]), (255, 32, 8, [90, 1000]),
    (128, 192, 24, [265, 21, 198]), (130, 80, 40, [265, 21, 198]), (128, 24, 24, [1, 2, 700, 31] * 4), (200, 64, 16, [40] * 16)])
def test_many_heads(dev, clean_status, N, Hq, Hkv, Ts):
    check(dev, Ts, N, Hq, Hkv, seed=43)


@pytest.mark.parametrize("seed", range(6))
def test_random_batches_on_one_workspace(dev, seed):
    """Any geometry, lengths, masks (also ones that leave rows empty) and requests
    without room in between, on one workspace: the formula's output, the same bits
    twice, and nothing written for a request without room."""
    import tree_verified_block_gb300 as g
    g.reset_device_status()
    gen = W.rng(71, seed)
    kg, vg, scale = 0.75, 5.5 / 2688, 128 ** -0.5
    ws = None
    for _ in range(8):
        B, Hkv, G = (int(gen.choice(c)) for c in ([1, 2, 3, 5, 16], [1, 2, 3, 8, 24], [1, 2, 4, 8]))
        N, hi = int(gen.choice([0, 1, 3, 7, 15, 16, 31, 63, 64, 100, 128, 200, 255])), int(gen.choice([2, 40, 300, 2000]))
        rows, Hq, hi = N + 1, G * Hkv, max(2, min(hi, 100000 // (B * Hkv)))
        caches, layers, trees, seens, Ts, room = [], [], [], [], [], []
        for _ in range(B):
            T = int(gen.integers(0, hi))
            cap = T + rows + (T + rows) % 2
            room.append(bool(gen.random() > 0.2))
            t_len = T if room[-1] else int(gen.choice([-1, cap - rows + 1, 2 ** 31 - 1]))
            t = random_tree(gen, N, 16, T)
            if N and gen.random() < 0.5:
                t["seen"] = np.tril(gen.random((rows, rows)) < gen.choice([0.02, 0.5, 0.98]))
                t["anc"] = anc_words(t["seen"])
            caches.append(random_cache(gen, Hkv, cap, kg, vg))
            layers.append(layer_of(g, caches[-1], torch.tensor([t_len], dtype=torch.int32, device=dev), dev, kg, vg))
            trees.append(upload_tree(g, t, 16, dev))
            seens.append(t["seen"])
            Ts.append(T)
        q = bf16_tensor(W.normal_bf16(gen, (B, rows, Hq, 128)), dev)
        need = g.kv4_tree_attention_workspace_bytes(rows, Hq, layers)
        if ws is None or ws.numel() < need:
            ws = g.workspace(need, dev)
        outs = [torch.full_like(q, 3.0) for _ in range(2)]
        for out in outs:
            g.kv4_tree_attention(q, layers, trees, scale, out, ws)
        what = (B, Hkv, G, N, Ts, room)
        assert g.device_status()[0] == (0 if all(room) else 2), what
        g.reset_device_status()
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16)), what
        for r in range(B):
            if room[r]:
                o, tol = attention64(q[r], caches[r], Ts[r], seens[r], scale, kg, vg, dev)
                assert torch.all((outs[0][r].double() - o).abs() <= tol), what
            else:
                assert torch.all(outs[0][r] == 3), what


@pytest.mark.parametrize("N", [2, 50])
def test_a_row_whose_scores_are_all_minus_infinity_is_not_a_number(dev, clean_status, N):
    import tree_verified_block_gb300 as g
    gen = W.rng(47)
    rows, T = N + 1, 300
    cache = random_cache(gen, 2, T + rows + (T + rows) % 2, 1.0, 1.0)
    cache[0][:, :, 2] = (cache[0][:, :, 2] & 0x0F) | 0x20  # element 5 of every K row is 1 (times a scale > 0)
    layer = layer_of(g, cache, torch.tensor([T], dtype=torch.int32, device=dev), dev)
    q = bf16_tensor(W.normal_bf16(gen, (1, rows, 8, 128)), dev)
    q[0, 1, 3, 5] = float("-inf")
    out = torch.zeros_like(q)
    g.kv4_tree_attention(q, [layer], [upload_tree(g, random_tree(gen, N, 8, T), 8, dev)], 0.09, out,
                         g.workspace(g.kv4_tree_attention_workspace_bytes(rows, 8, [layer]), dev))
    hit = torch.zeros(rows, 8, dtype=torch.bool, device=dev)
    hit[1, 3] = True
    assert torch.equal(out[0].isnan().all(-1), hit) and torch.equal(out[0].isnan().any(-1), hit)


def test_rows_read_back_are_the_next_call_s_prefix(dev, clean_status):
    """kv4_read_rows into a 16-bit cache, then tree attention over it, which
    loads prefix slots as early as it may: the new ones every time."""
    import tree_verified_block_gb300 as g
    gen = W.rng(53)
    N, Hq, Hkv, T = 15, 8, 2, 6000
    rows = N + 1
    tree = upload_tree(g, random_tree(gen, N, 8, T), 8, dev)
    t_len = torch.tensor([T], dtype=torch.int32, device=dev)
    sources = [g.Views([layer_of(g, random_cache(gen, Hkv, T + rows, 1.0, 1.0), t_len, dev)]) for _ in range(4)]
    dst = torch.zeros(1, 2, Hkv, T + rows, 128, dtype=torch.bfloat16, device=dev)
    kv = g.KVLayer(dst[0, 0], dst[0, 1], t_len)
    q = bf16_tensor(W.normal_bf16(gen, (rows, Hq, 128)), dev)
    ws = g.workspace(g.tree_attention_workspace_bytes(rows, Hq, kv), dev)
    outs = [[torch.zeros_like(q) for _ in sources] for _ in range(2)]
    for wait in (1, 0):
        for s, out in zip(sources, outs[wait]):
            g.kv4_read_rows(s, 0, T + rows, dst)
            if wait:
                torch.cuda.synchronize()
            g.tree_attention(q, kv, tree, 0.09, out, ws)
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_a_prompt_s_rows_are_the_next_call_s_prefix(dev, clean_status):
    """qk_norm_rope of a prompt into slots 0.., then tree attention whose T
    counts those slots already: it must see them as written."""
    import tree_verified_block_gb300 as g
    gen = W.rng(59)
    N, Hq, Hkv, T = 15, 8, 2, 4000
    rows = N + 1
    tree = upload_tree(g, random_tree(gen, N, 8, T), 8, dev)
    k, v = (torch.zeros(Hkv, T + rows, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    zero = torch.zeros(1, dtype=torch.int32, device=dev)
    prompt, kv = g.KVLayer(k, v, zero), g.KVLayer(k, v, torch.tensor([T], dtype=torch.int32, device=dev))
    xs = [bf16_tensor(W.normal_bf16(gen, (T + rows, (Hq + 2 * Hkv) * 128)), dev) for _ in range(4)]
    pos = torch.arange(T + rows, dtype=torch.int32, device=dev)[None]
    rope = g.Rope(128, 1e4)
    q_out = torch.zeros(T + rows, Hq, 128, dtype=torch.bfloat16, device=dev)
    q = bf16_tensor(W.normal_bf16(gen, (rows, Hq, 128)), dev)
    ws = g.workspace(g.tree_attention_workspace_bytes(rows, Hq, kv), dev)
    outs = [[torch.zeros_like(q) for _ in xs] for _ in range(2)]
    for wait in (1, 0):
        for x, out in zip(xs, outs[wait]):
            g.qk_norm_rope(x, Hq, None, None, 1e-6, pos, rope, q_out, prompt)
            if wait:
                torch.cuda.synchronize()
            g.tree_attention(q, kv, tree, 0.09, out, ws)
    torch.cuda.synchronize()
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def run_cases(lib, out):
    r = subprocess.run([sys.executable, os.path.join(HERE, "_checked_kv4_cases.py"), lib, out], capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-4000:]
    return np.load(out)


def test_checked_build_matches_and_reports_nothing(tmp_path):
    checked = os.path.join(LIB_DIR, "libglance_check.so")
    if not os.path.exists(checked):
        pytest.skip("libglance_check.so not built (run __graft_entry__.build())")
    normal = run_cases(os.path.join(LIB_DIR, "libglance.so"), str(tmp_path / "normal.npz"))
    chk = run_cases(checked, str(tmp_path / "checked.npz"))
    assert sorted(normal.files) == sorted(chk.files)
    assert np.all(chk["status"] == 0), chk["status"]
    for k in normal.files:
        assert np.array_equal(normal[k], chk[k], equal_nan=True), k
