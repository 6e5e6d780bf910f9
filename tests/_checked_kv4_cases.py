"""Runs a fixed set of small calls on 4-bit caches and of norm + rotary rows
through one build of the library and saves every output:
`python tests/_checked_kv4_cases.py LIB OUT.npz`. test_gpu_kv4_mixed.py runs it
once with libglance.so and once with the bounds-checked libglance_check.so and
compares the two. Inputs are seeded."""
import os
import sys

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, os.path.dirname(HERE))
sys.path.insert(0, HERE)

import tree_verified_block_gb300._binding as b  # noqa: E402

b.LIB_PATH = sys.argv[1]

import torch  # noqa: E402

import tree_verified_block_gb300 as g  # noqa: E402
import workloads as W  # noqa: E402
from _kv4_util import bytes_of, random_tree, up, upload_tree  # noqa: E402


def bf16(bits, dev):
    return torch.from_numpy(bits.view(np.int16)).to(dev).view(torch.bfloat16)


def main(out_path):
    dev = torch.device("cuda:0")
    torch.cuda.set_device(dev)
    res = {}
    gen = W.rng(31)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device=dev)
    # caches that are exactly as long as the call needs (T + rows = t_cap), one
    # kv head behind the other: few and many query rows, one and several requests
    for N, Hq, Hkv, Ts in ((0, 8, 2, [399, 7]), (3, 8, 2, [60]), (11, 2, 2, [1012, 0, 300]), (63, 8, 2, [960, 64]), (130, 2, 1, [397])):
        rows = N + 1
        layers, trees, t_lens = [], [], []
        for T in Ts:
            cap = T + rows + (T + rows) % 2
            t_lens.append(torch.tensor([cap - rows], dtype=torch.int32, device=dev))
            layers.append(g.KV4Layer.empty(Hkv, cap, i32(1), 0.5, 0.01))
            g.kv4_write_rows(bf16(W.normal_bf16(gen, (1, 2, Hkv, cap, 128)), dev), [layers[-1]], cap)
            layers[-1] = g.KV4Layer(layers[-1].k, layers[-1].k_scale, layers[-1].v, layers[-1].v_scale, t_lens[-1], 0.5, 0.01)
            trees.append(random_tree(gen, N, 8, T))
        q = bf16(W.normal_bf16(gen, (len(Ts), rows, Hq, 128)), dev)
        out = torch.zeros_like(q)
        ups = [upload_tree(g, t, 8, dev) for t in trees]
        ws = g.workspace(g.kv4_tree_attention_workspace_bytes(rows, Hq, layers), dev)
        g.kv4_tree_attention(q, layers, ups if N else None, 128 ** -0.5, out, ws)
        key = f"{N}_{Hq}_{len(Ts)}"
        res["out_" + key] = out.view(torch.int16).cpu().numpy()
        if N:
            arg = up(np.stack([gen.permutation(t["token"]).astype(np.int32) for t in trees]), dev)
            for r, t in enumerate(trees):  # the path to the last row
                u = N
                while t["parent"][u] >= 0:
                    arg[r, int(t["parent"][u])] = int(t["token"][u])
                    u = t["parent"][u]
            n_acc, tok, root = i32(len(Ts)), i32(len(Ts), 8), i32(len(Ts))
            g.kv4_accept_commit(ups, arg, layers, n_acc, tok, root, g.workspace(256, dev))
            res["commit_" + key] = torch.cat([n_acc, tok.view(-1), root, *t_lens]).cpu().numpy()
        back = torch.zeros(1, 2, Hkv, layers[0].k.shape[1], 128, dtype=torch.bfloat16, device=dev)
        g.kv4_read_rows([layers[0]], 0, back.shape[3], back)
        res["back_" + key] = back.view(torch.int16).cpu().numpy()
        for r, l in enumerate(layers):
            for i, x in enumerate(bytes_of(l)):
                res[f"bytes_{key}_{r}_{i}"] = x
    for dtype, D, M in ((torch.bfloat16, 128, 37), (torch.float32, 64, 5)):
        x = torch.from_numpy(gen.standard_normal((2 * M, 8 * D)).astype(np.float32)).to(dev, dtype)
        kvs = [g.KVLayer(torch.zeros(2, M + 3, D, dtype=dtype, device=dev), torch.zeros(2, M + 3, D, dtype=dtype, device=dev),
                         torch.full((1,), 3, dtype=torch.int32, device=dev)) for _ in range(2)]
        w = torch.from_numpy(gen.uniform(0.5, 1.5, D).astype(np.float32)).to(dev)
        pos = up(gen.integers(-5, 1 << 20, (2, 2 * M)).astype(np.int32), dev)
        q = torch.zeros(2 * M, 4, D, dtype=dtype, device=dev)
        g.qk_norm_rope(x, 4, w, w, 1e-6, pos, g.Rope(D, 1e4, [D // 4, D // 4]), q, kvs)
        for i, t in enumerate([q] + [c for l in kvs for c in (l.k, l.v)]):
            res[f"rope_{D}_{i}"] = t.float().cpu().numpy()
    st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
    g.get_status(st)
    torch.cuda.synchronize()
    res["status"] = st.cpu().numpy()
    np.savez(out_path, **res)


if __name__ == "__main__":
    main(sys.argv[2])
