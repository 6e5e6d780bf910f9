"""Shared helpers of the 4-bit cache tests: caches on the device beside their
bytes on the host, random packed trees, attention in 64 bits."""
import numpy as np
import torch

import workloads as W
from oracle import kv4 as okv4


def up(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def random_cache(gen, Hkv, slots, k_global, v_global, std=1.0):
    """Bytes (k, k_scale, v, v_scale) of quantised N(0, std^2) rows."""
    out = []
    for g in (k_global, v_global):
        x = W.bf16_bits_to_f32(W.normal_bf16(gen, (Hkv, slots, 128), std))
        codes, scale = okv4.quantise(x, g)
        out += [okv4.pack(codes), scale]
    return out


def layer_of(g, cache, t_len, dev, k_global=1.0, v_global=1.0, t_cap=None):
    """A KV4Layer on copies of the bytes; t_cap below the slots leaves a gap between heads."""
    n = cache[0].shape[1] if t_cap is None else t_cap
    t = [up(c, dev)[:, :n] for c in cache]
    return g.KV4Layer(*t, t_len, k_global, v_global)


def bytes_of(layer):
    return [t.cpu().numpy() for t in (layer.k, layer.k_scale, layer.v, layer.v_scale)]


def random_tree(rng, N, L, T=0, chain=False):
    """Host arrays of a packed tree of N + 1 rows (breadth first, sibling tokens distinct)."""
    parent, depth = [-1], [0]
    while len(parent) <= N:
        i = len(parent)
        ok = [p for p in range(max(0, parent[-1]), i) if depth[p] < L]
        p = i - 1 if chain else ok[min(int(rng.integers(0, 3)), len(ok) - 1)]
        parent.append(p)
        depth.append(depth[p] + 1)
    rows = N + 1
    order = sorted(range(rows), key=lambda i: depth[i])
    place = {o: i for i, o in enumerate(order)}
    parent = np.array([-1 if parent[o] < 0 else place[parent[o]] for o in order], dtype=np.int32)
    depth = np.array([depth[o] for o in order], dtype=np.int32)
    seen = np.zeros((rows, rows), dtype=bool)
    for i in range(rows):
        if parent[i] >= 0:
            seen[i] = seen[parent[i]]
        seen[i, i] = True
    token = rng.permutation(50000)[:rows].astype(np.int32)
    return dict(token=token, parent=parent, depth=depth, pos_id=(T + depth).astype(np.int32), seen=seen,
                anc=anc_words(seen))


def anc_words(seen):
    rows = seen.shape[0]
    words = np.zeros((rows, (rows + 63) // 64), dtype=np.uint64)
    for i, k in zip(*np.nonzero(seen)):
        words[i, k // 64] |= np.uint64(1) << np.uint64(k % 64)
    return words


def upload_tree(g, t, L, dev):
    out = g.Tree(len(t["token"]) - 1, L, dev)
    for name in ("token", "parent", "depth", "pos_id"):
        getattr(out, name).copy_(up(t[name], dev))
    out.anc.copy_(up(t["anc"].view(np.int64), dev))
    return out


def attention64(q, cache, T, seen, scale, k_global, v_global, dev):
    """(out, tolerance) of one request in 64 bits on the device: q bf16 tensor
    [rows][Hq][128], cache the host bytes, seen bool [rows][rows].

    Tolerance, from the roundings the call has: the output to bf16, 2^-8 |o|
    (half a step); the softmax weights to f16, half a step 2^-11 of each, or
    2^-25 absolute where they are below 2^-14 of the running maximum; scores in
    fp32, 132 terms of at most 2^-23 each (products and partial sums; the
    tensor unit may truncate, a whole step) of sum |q| |k| * scale, which moves
    a weight by that much and the sum of weights as well; 2^-20 for the
    exponential and the rest of the fp32 arithmetic."""
    rows, Hq, _ = q.shape
    Hkv, n = cache[0].shape[0], T + rows
    G = Hq // Hkv
    k = up(okv4.values(cache[0][:, :n], cache[1][:, :n], k_global), dev)
    v = up(okv4.values(cache[2][:, :n], cache[3][:, :n], v_global), dev)
    x = q.double().view(rows, Hkv, G, 128).permute(1, 2, 0, 3)
    vis = torch.cat((torch.ones(rows, T, dtype=torch.bool), torch.from_numpy(seen)), 1).to(dev)
    k0, v0 = k.nan_to_num(), v.nan_to_num()
    s = (torch.einsum("hgrd,hkd->hgrk", x, k0) * scale).masked_fill(~vis, -torch.inf)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(m > -torch.inf, m, torch.zeros_like(m)))
    l = p.sum(-1, keepdim=True)
    p = torch.where(l > 0, p / torch.where(l > 0, l, torch.ones_like(l)), torch.zeros_like(p))
    o = torch.einsum("hgrk,hkd->hgrd", p, v0)
    ds = torch.einsum("hgrd,hkd->hgrk", x.abs(), k0.abs()).masked_fill(~vis, 0).amax(-1, keepdim=True) * scale * 132 * 2 ** -23
    spread = torch.einsum("hgrk,hkd->hgrd", p, v0.abs())
    tol = 2 ** -8 * o.abs() + spread * (2 * 2 ** -11 + 2 * ds + 2 ** -20) + n * 2 ** -25 * v0.abs().amax((1, 2))[:, None, None, None]
    back = lambda t: t.permute(2, 0, 1, 3).reshape(rows, Hq, 128)
    return back(o), back(tol)
