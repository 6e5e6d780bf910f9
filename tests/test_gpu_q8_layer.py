"""A verify round with the target's layer in 8 bits, as a user runs it: norm
rows, projections, rotary rows, tree attention, the LM head's logits, the draw
and the walk, in one captured graph; and each step against its own definition on
the values that the step before it left."""
import numpy as np
import pytest
import torch

from oracle import q8
from oracle.truncated_sampling import sample_row
from oracle.walk import walk as o_walk
from test_gpu_attention import random_tree, upload_tree

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def f64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("N", [0, 31, 70])
def test_a_sampled_round_in_8_bits(dev, clean_status, N):
    import tree_verified_block_gb300 as g
    d, inter, Hq, Hkv, V, T, L = 512, 1152, 4, 2, 5003 // 8 * 8, 90, 7
    M = N + 1
    gen = torch.Generator(device=dev).manual_seed(N)
    rn = lambda *s: torch.randn(*s, generator=gen, device=dev)

    def weights(rows, width):
        codes, scales = torch.zeros(rows, width, dtype=torch.uint8, device=dev), torch.zeros(rows, device=dev)
        g.q8_rows(rn(rows, width) * width ** -0.5, codes, scales)
        return codes, scales

    wqkv, wo, wgu, wdown, whead = weights((Hq + 2 * Hkv) * 128, d), weights(d, Hq * 128), weights(2 * inter, d), weights(d, inter), weights(V, d)
    g1, g2, g3 = (1 + 0.1 * rn(d) for _ in range(3))
    x = rn(M, d).to(BF)
    ref = random_tree(max(N, 1), L, T, 3)
    tree = upload_tree(ref, L, dev)
    t_len = torch.tensor([T], dtype=torch.int32, device=dev)
    kv = g.KVLayer(rn(Hkv, T + M + 4, 128).to(BF), rn(Hkv, T + M + 4, 128).to(BF), t_len)
    pos = (tree.pos_id if N else torch.full((1,), T, dtype=torch.int32, device=dev))
    nxt = pos + 1
    qkv, q, att = torch.zeros(M, (Hq + 2 * Hkv) * 128, dtype=BF, device=dev), *(torch.zeros(M, Hq, 128, dtype=BF, device=dev) for _ in range(2))
    c, s = torch.zeros(M, d, dtype=torch.uint8, device=dev), torch.zeros(M, device=dev)
    ca, sa = torch.zeros(M, inter, dtype=torch.uint8, device=dev), torch.zeros(M, device=dev)
    act, h, total = torch.zeros(M, inter, dtype=BF, device=dev), torch.zeros(M, d, dtype=BF, device=dev), torch.zeros(M, d, dtype=BF, device=dev)
    mlp, out = torch.zeros(M, d, dtype=BF, device=dev), torch.zeros(M, d, dtype=BF, device=dev)
    logits, tokens, gap = torch.zeros(M, V, device=dev), torch.zeros(M, dtype=torch.int32, device=dev), torch.zeros(M, device=dev)
    row = lambda v, dt=torch.float32: torch.full((M,), v, dtype=dt, device=dev)
    temperature, top_k, top_p = row(0.8), row(40, torch.int32), row(0.9)
    rope = g.Rope(128, 1e6)
    ws = g.workspace(g.tree_attention_workspace_bytes(M, Hq, kv) if N else 0, dev)
    n_acc, acc, root = (torch.zeros(n, dtype=torch.int32, device=dev) for n in (1, L, 1))
    wsc = g.workspace(g.accept_commit_workspace_bytes(1), dev)

    def rnd():
        g.q8_norm_rows(x, None, g1, 1e-6, None, c, s)
        g.q8_linear(c, s, *wqkv, qkv)
        g.qk_norm_rope(qkv, Hq, None, None, 1e-6, pos[None], rope, q, kv)
        if N:
            g.tree_attention(q, kv, tree, 128 ** -0.5, att, ws)
        else:
            att.copy_(q)
        g.q8_rows(att.view(M, -1), c, s)
        g.q8_linear(c, s, *wo, h, residual=x)
        g.q8_norm_rows(h, None, g2, 1e-6, None, c, s)
        g.q8_linear(c, s, *wgu, act, act="silu", gated=True)
        g.q8_rows(act, ca, sa)
        g.q8_linear(ca, sa, *wdown, mlp)
        g.q8_norm_rows(mlp, h, g3, 1e-6, out, c, s)
        g.q8_linear(c, s, *whead, logits)
        g.sample(logits, temperature, top_k, top_p, None, 99, nxt, None, tokens, gap)

    stream = torch.cuda.Stream(dev)
    rnd()
    torch.cuda.synchronize()
    first = [t.clone() for t in (qkv, h, act, out, logits, tokens, gap)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        rnd()
        if N:
            g.accept_commit(tree, tokens, [kv], n_acc, acc, root, wsc)
    for t in (qkv, h, act, out, logits, tokens):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((qkv, h, act, out, logits, tokens, gap), first))

    val = lambda p: q8.code_values(p[0].cpu().numpy()) * f64(p[1])[:, None]
    # the round's end, from what it left: codes of the last norm, logits, tokens
    assert torch.equal(out, (mlp.float() + h.float()).to(BF))
    want, _, size = q8.linear(val((c, s)), val(whead))
    assert np.all(np.abs(f64(logits) - want) <= (d / 16 + 20) * 2.0 ** -23 * size)
    for i in range(M):
        token, _, near = sample_row(f64(logits)[i], 99, int(nxt[i]), 0, 0.8, 40, 0.9)
        assert near < 2.0 ** -21 or int(tokens[i]) == token
    a8, _, size = q8.linear(val((ca, sa)), val(wdown))
    assert np.all(np.abs(f64(mlp) - a8) <= 2.0 ** -8 * np.abs(a8) + (inter / 16 + 20) * 2.0 ** -23 * size)
    # the layer against the same in 64 bits without 8-bit rows: e4m3's half step
    # of 2^-4 is 0.026 of a value in the mean (uniform in its steps), two such
    # factors in each product, norms and activations of slope about 1, three
    # products one after the other: about 0.04 * sqrt(3), and four times that
    y = q8.norm_rows(f64(x), f64(g1), 1e-6) @ val(wqkv).T
    assert np.linalg.norm(f64(qkv) - y) <= 4 * 0.04 * np.linalg.norm(y)
    hh = f64(h)
    gu = q8.norm_rows(hh, f64(g2), 1e-6) @ val(wgu).T
    a = q8.activate(gu[:, :inter], "silu") * gu[:, inter:]
    assert np.linalg.norm(f64(act) - a) <= 4 * 0.07 * np.linalg.norm(a)
    if N:
        n, path, toks, nr = o_walk(ref, tokens.cpu().numpy(), L)
        assert int(n_acc) == n and int(root) == nr and acc[:n].tolist() == list(toks)[:n] and int(t_len) == T + n + 1
