"""Operators around a 4-bit K/V cache: the cases that are measured.

Four operators of the verify path are listed, each in a plain form (elementary
torch operations in 32 bits) and as a user of the library calls it:

* ``rope``       RMS norm of every query and key head and the rotary position
                 (one axis, or time / height / width) in one pass; q to a
                 buffer, k and v into the layer's cache;
* ``rows``       rows of K and V written into 4-bit caches, and read back;
* ``attention``  tree attention (one row: plain decoding) over 4-bit caches;
* ``round``      the end of a verify round on 4-bit caches: the tree rows go
                 in, the walk commits the accepted path, the rows are read.

A 4-bit cache holds, per layer and kv head and slot, 128 codes of 4 bits
(sign, two exponent bits, one fraction bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6; the
even element of a byte in its low half) and 8 scales of 8 bits (e4m3), one per
16 elements. An element stands for code * scale * global, with one global
factor for K and one for V.
"""
import math
import random

import torch

own = False
DEV = "cuda"
D = 128
GROUP = 16
#: What the eight magnitudes of a 4-bit code stand for.
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # the 64 packed rows of one verify layer (32 / 8 heads), text positions far into a long context
        dict(name="rope verify rows", op="rope", M=64, T=4096, Hq=32, Hkv=8, D=128, dtype="bf16", axes=1,
             interleaved=False, norm=True, theta=1e6, pos_hi=131072),
        # a prompt of several images and a video: three axes, interleaved frequencies; an odd number of rows
        dict(name="rope image prompt", op="rope", M=16383, T=0, Hq=32, Hkv=8, D=128, dtype="bf16", axes=3,
             interleaved=True, norm=True, theta=1e6, pos_hi=4096),
        # the fp32 target of the exactness tests: head_dim 32, no norm, chunked axes
        dict(name="rope fp32 rows", op="rope", M=777, T=13, Hq=4, Hkv=2, D=32, dtype="f32", axes=2,
             interleaved=False, norm=False, theta=1e4, pos_hi=2048),
        # the tree rows of all 36 layers, written at once and read back
        dict(name="rows tree 36 layers", op="rows", layers=36, rows=64, T=4096, Hkv=8, unit=False),
        # a long prompt's K/V moved into 4 bits, an odd number of rows at an odd slot
        dict(name="rows prompt", op="rows", layers=12, rows=8191, T=5, Hkv=8, unit=True),
        # one new token of one request after a short prompt: latency
        dict(name="decode 1 x 1000", op="attention", B=1, N=0, T_lo=1000, T_hi=1000, Hq=32, Hkv=8),
        # one new token each of 16 requests of mixed length
        dict(name="decode 16 x 512..32768", op="attention", B=16, N=0, T_lo=512, T_hi=32768, Hq=32, Hkv=8),
        # a verify round's layer: 63 candidates
        dict(name="verify 63 at 4096", op="attention", B=1, N=63, T_lo=4096, T_hi=4096, Hq=32, Hkv=8),
        # the same for a ragged batch of 8 requests
        dict(name="verify 63 x 8 ragged", op="attention", B=8, N=63, T_lo=512, T_hi=8192, Hq=32, Hkv=8),
        # a very long context: the largest case
        dict(name="verify 63 at 131072", op="attention", B=1, N=63, T_lo=131072, T_hi=131072, Hq=32, Hkv=8),
        # the end of a round over 36 layers, one request
        dict(name="round 36 layers", op="round", B=1, N=63, L=15, layers=36, T=4096, Hkv=8),
        # the same for a batch, shallow layers, a wide tree
        dict(name="round 8 requests", op="round", B=8, N=255, L=15, layers=6, T=1111, Hkv=4),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rows", "attention", "attention", "round"))
    Hkv = rng.choice((1, 2, 4, 8))
    if op == "rope":
        dtype = rng.choice(("bf16", "bf16", "f32"))
        axes = rng.choice((1, 2, 3))
        return dict(op=op, M=_log_int(rng, 1, 16383 if dtype == "bf16" else 8000), T=rng.randrange(0, 600),
                    Hq=Hkv * rng.choice((1, 2, 4)), Hkv=Hkv, D=rng.choice((32, 64, 128)), dtype=dtype, axes=axes,
                    interleaved=axes > 1 and rng.random() < 0.5, norm=rng.random() < 0.7,
                    theta=rng.choice((1e4, 1e6, 5e6)), pos_hi=_log_int(rng, 64, 1 << 20))
    if op == "rows":
        layers = rng.randrange(1, 37)
        return dict(op=op, layers=layers, rows=_log_int(rng, 1, min(8191, 12 * 8191 // layers)),
                    T=rng.randrange(0, 3000), Hkv=Hkv, unit=rng.random() < 0.5)
    if op == "round":
        return dict(op=op, B=rng.randrange(1, 9), N=rng.randrange(1, 256), L=rng.randrange(3, 17),
                    layers=rng.randrange(1, 7), T=rng.randrange(0, 5000), Hkv=Hkv)
    B = rng.choice((1, 1, 2, 5, 8, 16))
    N = rng.choice((0, 0, _log_int(rng, 1, 255), _log_int(rng, 1, 255)))
    Hq = Hkv * rng.choice((1, 2, 4, 8))
    hi = 131072 * 64 * 32 // (B * (N + 1) * Hq)
    hi = _log_int(rng, 1, max(2, min(131072 // B, hi)))
    return dict(op=op, B=B, N=N, T_lo=max(0, hi // rng.choice((1, 2, 16)) - 1), T_hi=hi, Hq=Hq, Hkv=Hkv)


def lengths(case):
    """The prefix length of every request, from T_lo to T_hi in equal ratios."""
    B, lo, hi = case["B"], case["T_lo"], case["T_hi"]
    if B == 1:
        return [hi]
    return [int(round((lo + 1) * ((hi + 1) / (lo + 1)) ** (r / (B - 1)))) - 1 for r in range(B)]


# --------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device=DEV) * std).to(dtype)


def _random_tree(rng, N, L):
    """(parent, depth, list of ancestor lists) of N + 1 rows in packed order, depth <= L."""
    parent, depth = [-1], [0]
    while len(parent) <= N:
        # breadth first with a bias to early rows, as the best-first trees have it
        p = min(int(len(parent) * rng.random() ** 1.5), len(parent) - 1)
        if depth[p] < L:
            parent.append(p)
            depth.append(depth[p] + 1)
    order = sorted(range(N + 1), key=lambda i: depth[i])
    # parents first by depth, then by the parent's own place
    place = {}
    out_parent, out_depth = [], []
    by_depth = {}
    for i in order:
        by_depth.setdefault(depth[i], []).append(i)
    for d in sorted(by_depth):
        for i in sorted(by_depth[d], key=lambda i: place.get(parent[i], -1)):
            place[i] = len(out_parent)
            out_parent.append(place[parent[i]] if parent[i] >= 0 else -1)
            out_depth.append(d)
    anc = []
    for i, p in enumerate(out_parent):
        anc.append(([] if p < 0 else anc[p]) + [i])
    return out_parent, out_depth, anc


def _tree_state(rng, N, L, T):
    parent, depth, anc = _random_tree(rng, N, L)
    rows = N + 1
    words = (rows + 63) // 64
    bits = [[0] * words for _ in range(rows)]
    seen = torch.zeros(rows, rows, dtype=torch.bool)
    for i, a in enumerate(anc):
        seen[i, a] = True
        for k in a:
            bits[i][k // 64] |= 1 << (k % 64)
    signed = [[w - (1 << 64) if w >> 63 else w for w in r] for r in bits]
    i32 = dict(dtype=torch.int32, device=DEV)
    token = rng.sample(range(151936), rows)
    return dict(token=torch.tensor(token, **i32), parent=torch.tensor(parent, **i32),
                depth=torch.tensor(depth, **i32), pos_id=torch.tensor([T + d for d in depth], **i32),
                anc=torch.tensor(signed, dtype=torch.int64, device=DEV), seen=seen.to(DEV), paths=anc)


def _empty_cache(Hkv, slots, *lead):
    u8 = dict(dtype=torch.uint8, device=DEV)
    return dict(k=torch.zeros(*lead, Hkv, slots, D // 2, **u8), k_scale=torch.zeros(*lead, Hkv, slots, D // GROUP, **u8),
                v=torch.zeros(*lead, Hkv, slots, D // 2, **u8), v_scale=torch.zeros(*lead, Hkv, slots, D // GROUP, **u8))


def _slots(n):
    return (n + 15) // 16 * 16


def prepare(case, seed):
    gen = _gen(seed)
    rng = random.Random(int(seed) * 1000003 + 17)
    op = case["op"]
    s = dict(case=case)
    if op == "rope":
        M, Hq, Hkv, Dh, T = case["M"], case["Hq"], case["Hkv"], case["D"], case["T"]
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["qkv"] = _normal(gen, M, (Hq + 2 * Hkv) * Dh, std=1.7, dtype=dt)
        s["q_norm"] = 1 + 0.2 * torch.randn(Dh, generator=gen, device=DEV) if case["norm"] else None
        s["k_norm"] = 1 + 0.2 * torch.randn(Dh, generator=gen, device=DEV) if case["norm"] else None
        s["pos"] = torch.randint(0, case["pos_hi"], (case["axes"], M), generator=gen, device=DEV, dtype=torch.int32)
        s["q_out"] = torch.zeros(M, Hq, Dh, dtype=dt, device=DEV)
        s["k"] = torch.zeros(Hkv, T + M + 9, Dh, dtype=dt, device=DEV)
        s["v"] = torch.zeros(Hkv, T + M + 9, Dh, dtype=dt, device=DEV)
        s["t_len"] = torch.tensor([T], dtype=torch.int32, device=DEV)
        s["sections"] = sections(case)
    elif op == "rows":
        n, rows, Hkv, T = case["layers"], case["rows"], case["Hkv"], case["T"]
        s["src"] = _normal(gen, n, 2, Hkv, rows, D, std=1.0)
        s["cache"] = _empty_cache(Hkv, _slots(T + rows), n)
        s["t_len"] = torch.tensor([T], dtype=torch.int32, device=DEV)
        s["dst"] = torch.zeros(n, 2, Hkv, rows, D, dtype=torch.bfloat16, device=DEV)
        # the factors of a calibrated cache: the largest value meets the largest code and scale
        s["k_global"], s["v_global"] = (1.0, 1.0) if case["unit"] else (6.1 / 2688, 5.7 / 2688)
    elif op == "attention":
        B, N, Hq, Hkv = case["B"], case["N"], case["Hq"], case["Hkv"]
        Ts = lengths(case)
        s["q"] = _normal(gen, B, N + 1, Hq, D)
        s["out"] = torch.zeros(B, N + 1, Hq, D, dtype=torch.bfloat16, device=DEV)
        s["trees"] = [_tree_state(rng, N, 16, T) for T in Ts]
        s["k_global"], s["v_global"] = 0.75, 5.5 / 2688
        s["caches"] = []
        for T in Ts:
            c = _empty_cache(Hkv, _slots(T + N + 1 + 64))
            n = T + N + 1
            for name, g in (("k", s["k_global"]), ("v", s["v_global"])):
                for h in range(Hkv):
                    codes, scale, _ = quantise(torch.randn(n, D, generator=gen, device=DEV).to(torch.bfloat16), g)
                    c[name][h, :n] = codes[..., 0::2] | codes[..., 1::2] << 4
                    c[name + "_scale"][h, :n] = scale.view(torch.uint8)
            s["caches"].append(c)
        s["t_len"] = [torch.tensor([T], dtype=torch.int32, device=DEV) for T in Ts]
    else:
        B, N, L, n, T, Hkv = case["B"], case["N"], case["L"], case["layers"], case["T"], case["Hkv"]
        s["trees"] = [_tree_state(rng, N, L, T + r) for r in range(B)]
        s["T"] = [T + r for r in range(B)]
        s["src"] = [_normal(gen, n, 2, Hkv, N + 1, D) for _ in range(B)]
        s["dst"] = [torch.zeros(n, 2, Hkv, N + 1, D, dtype=torch.bfloat16, device=DEV) for _ in range(B)]
        s["caches"] = [_empty_cache(Hkv, _slots(T + r + N + 1), n) for r in range(B)]
        s["k_global"], s["v_global"] = 1.0, 0.25
        argmax = torch.randint(151936, 200000, (B, N + 1), generator=gen, device=DEV, dtype=torch.int32)
        for r, t in enumerate(s["trees"]):
            path = t["paths"][rng.randrange(N + 1)]  # the target follows the tree to this row
            token = t["token"].tolist()
            for a, b in zip(path, path[1:]):
                argmax[r, a] = token[b]
        s["argmax"] = argmax
        s["t_len"] = torch.tensor(s["T"], dtype=torch.int32, device=DEV)
        s["t_start"] = s["t_len"].clone()
        s["n_accepted"] = torch.zeros(B, dtype=torch.int32, device=DEV)
        s["accepted"] = torch.zeros(B, L, dtype=torch.int32, device=DEV)
        s["new_root"] = torch.zeros(B, dtype=torch.int32, device=DEV)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The views, plans and workspaces that a user's program keeps."""
    import tree_verified_block_gb300 as g
    case, op = s["case"], s["case"]["op"]
    if op == "rope":
        s["rope"] = g.Rope(case["D"], case["theta"], s["sections"], case["interleaved"])
        s["kv"] = g.KVLayer(s["k"], s["v"], s["t_len"])
        return
    if "trees" in s:
        L = case.get("L", 16)
        trees = []
        for t in s["trees"]:
            tree = g.Tree(case["N"], L, DEV)
            for name in ("token", "parent", "depth", "pos_id", "anc"):
                getattr(tree, name).copy_(t[name])
            trees.append(tree)
        s["c_trees"] = g.Views(trees)
    kg, vg = s["k_global"], s["v_global"]
    if op == "rows":
        c = s["cache"]
        s["views"] = g.Views([g.KV4Layer(c["k"][i], c["k_scale"][i], c["v"][i], c["v_scale"][i], s["t_len"], kg, vg)
                              for i in range(case["layers"])])
    elif op == "attention":
        s["views"] = g.Views([g.KV4Layer(c["k"], c["k_scale"], c["v"], c["v_scale"], t, kg, vg)
                              for c, t in zip(s["caches"], s["t_len"])])
        s["ws"] = g.workspace(g.kv4_tree_attention_workspace_bytes(case["N"] + 1, case["Hq"], s["views"]), DEV)
    else:
        per = [g.Views([g.KV4Layer(c["k"][i], c["k_scale"][i], c["v"][i], c["v_scale"][i], s["t_len"][r:r + 1], kg, vg)
                        for i in range(case["layers"])]) for r, c in enumerate(s["caches"])]
        s["views"] = per
        s["all_views"] = g.Views([v for p in per for v in p])
        s["ws"] = g.workspace(g.kv4_accept_commit_workspace_bytes(case["B"], case["layers"]), DEV)


# ---------------------------------------------------------------- plain forms

def sections(case):
    """How many of the D / 2 frequencies each axis turns."""
    half, axes = case["D"] // 2, case["axes"]
    if axes == 1:
        return [half]
    rest = half // (axes + 1) + (1 if axes == 3 and half == 64 else 0)
    if case["interleaved"]:
        rest = min(rest, half // axes)
    if half == 64 and axes == 3:
        rest = 20
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def frequency_axis(case):
    """The axis of each frequency: runs, or taken in turn while an axis has some left (else the first)."""
    half, axes, sec = case["D"] // 2, case["axes"], sections(case)
    if not case["interleaved"]:
        return [a for a in range(axes) for _ in range(sec[a])]
    return [j % axes if j % axes and j // axes < sec[j % axes] else 0 for j in range(half)]


def quantise(x, g):
    """(codes, scales as e4m3, the values they stand for) of rows [..., 128]."""
    t = x.float().div_(g).unflatten(-1, (D // GROUP, GROUP))
    scale = (t.abs().amax(-1) / 6).clamp(max=448).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    y = torch.where(s > 0, t / s, torch.zeros_like(t))
    a = y.abs()
    m = (a > 0.25).byte()
    m += a >= 0.75
    m += a > 1.25
    m += a >= 1.75
    m += a > 2.5
    m += a >= 3.5
    m += a > 5
    codes = (m | (y < 0).byte() << 3).flatten(-2)
    value = torch.tensor(MAGNITUDES, device=x.device)[m.long()]
    value = (torch.where(y < 0, -value, value) * s * g).flatten(-2)
    return codes, scale, value


def decode(packed, scale, g):
    """The values of packed codes [..., 64] with scales [..., 8]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=packed.device)
    x = torch.stack((table[(packed & 15).long()], table[(packed >> 4).long()]), -1).flatten(-2)
    s = scale.view(torch.float8_e4m3fn).float()
    return (x.unflatten(-1, (D // GROUP, GROUP)) * s.unsqueeze(-1)).flatten(-2) * g


def _plain_rope(s):
    c = s["case"]
    M, Hq, Hkv, Dh, T = c["M"], c["Hq"], c["Hkv"], c["D"], c["T"]
    x = s["qkv"].float().view(M, Hq + 2 * Hkv, Dh)

    def norm(y, w):
        return y if w is None else y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * w

    j = torch.arange(Dh // 2, device=DEV, dtype=torch.float64)
    freq = c["theta"] ** (-2 * j / Dh)
    angle = s["pos"].double()[torch.tensor(frequency_axis(c), device=DEV)].t() * freq
    cos, sin = angle.cos().float().unsqueeze(1), angle.sin().float().unsqueeze(1)

    def turn(y):
        a, b = y[..., :Dh // 2], y[..., Dh // 2:]
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)

    s["q_out"].copy_(turn(norm(x[:, :Hq], s["q_norm"])))
    s["k"][:, T:T + M] = turn(norm(x[:, Hq:Hq + Hkv], s["k_norm"])).transpose(0, 1).to(s["k"].dtype)
    s["v"][:, T:T + M] = x[:, Hq + Hkv:].transpose(0, 1).to(s["v"].dtype)
    return [s["q_out"], s["k"], s["v"]]


def _plain_rows(s):
    k = quantise(s["src"][:, 0], s["k_global"])[2]
    v = quantise(s["src"][:, 1], s["v_global"])[2]
    return torch.stack((k, v), 1).to(torch.bfloat16)


def _plain_attention_one(q, c, seen, T, kg, vg, Hkv):
    rows, Hq = q.shape[0], q.shape[1]
    n = T + rows
    k = decode(c["k"][:, :n], c["k_scale"][:, :n], kg)
    v = decode(c["v"][:, :n], c["v_scale"][:, :n], vg)
    x = q.float().view(rows, Hkv, Hq // Hkv, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    sc = torch.bmm(x, k.transpose(1, 2)) * D ** -0.5
    visible = torch.cat((seen.new_ones(rows, T), seen), 1)
    sc = sc.view(Hkv, Hq // Hkv, rows, n).masked_fill_(~visible, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True))
    o = torch.bmm(p.view(Hkv, -1, n), v).view(Hkv, Hq // Hkv, rows, D) / p.sum(-1, keepdim=True)
    return o.permute(2, 0, 1, 3).reshape(rows, Hq, D)


def _plain_attention(s):
    case = s["case"]
    got = [_plain_attention_one(q, c, t["seen"], T, s["k_global"], s["v_global"], case["Hkv"])
           for q, c, t, T in zip(s["q"], s["caches"], s["trees"], lengths(case))]
    s["out"].copy_(torch.stack(got))
    return s["out"]


def _plain_round_one(t, src, dst, argmax, T, kg, vg):
    rows = argmax.numel()
    k, v = quantise(src[:, 0], kg)[2], quantise(src[:, 1], vg)[2]
    vals = torch.stack((k, v), 1).to(torch.bfloat16)
    up = t["parent"].clamp(min=0).long()
    fits = (argmax[up] == t["token"]) | (t["parent"] < 0)
    on_path = (fits | ~t["seen"]).all(1)
    depth = torch.where(on_path, t["depth"], torch.full_like(t["depth"], -1))
    a, last = depth.max(0)
    at = torch.arange(rows, device=DEV)
    slot = torch.full((rows + 1,), -1, device=DEV, dtype=torch.long)
    slot = slot.scatter(0, torch.where(on_path, t["depth"].long(), torch.full_like(at, rows)), at)[:rows]
    source = torch.where(at <= a, slot, at)
    dst.copy_(vals.index_select(3, source))
    tok = torch.where((at > 0) & (at <= a), t["token"][source], torch.zeros_like(t["token"]))[1:]
    return a, tok, argmax[last], T + a + 1


def _plain_round(s):
    got = [_plain_round_one(t, x, d, m, T, s["k_global"], s["v_global"])
           for t, x, d, m, T in zip(s["trees"], s["src"], s["dst"], s["argmax"], s["T"])]
    a = torch.stack([g[0] for g in got]).int()
    L = s["case"]["L"]
    tok = torch.stack([torch.cat((g[1], g[1].new_zeros(L)))[:L] for g in got])
    return [a, tok, torch.stack([g[2] for g in got]), torch.stack([g[3] for g in got]).int()] + s["dst"]


# ------------------------------------------------------------------------ run

def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"rope": _plain_rope, "rows": _plain_rows, "attention": _plain_attention, "round": _plain_round}[op](s)
    import tree_verified_block_gb300 as g
    if op == "rope":
        g.qk_norm_rope(s["qkv"], case["Hq"], s["q_norm"], s["k_norm"], 1e-6, s["pos"], s["rope"], s["q_out"], s["kv"])
        return [s["q_out"], s["k"], s["v"]]
    if op == "rows":
        g.kv4_write_rows(s["src"], s["views"], case["rows"])
        g.kv4_read_rows(s["views"], case["T"], case["rows"], s["dst"])
        return s["dst"]
    if op == "attention":
        g.kv4_tree_attention(s["q"], s["views"], s["c_trees"], D ** -0.5, s["out"], s["ws"])
        return s["out"]
    s["t_len"].copy_(s["t_start"])
    rows = case["N"] + 1
    for src, views in zip(s["src"], s["views"]):
        g.kv4_write_rows(src, views, rows)
    g.kv4_accept_commit(s["c_trees"], s["argmax"], s["all_views"], s["n_accepted"], s["accepted"], s["new_root"], s["ws"])
    for dst, views, T in zip(s["dst"], s["views"], s["T"]):
        g.kv4_read_rows(views, T, rows, dst)
    return [s["n_accepted"], s["accepted"], s["new_root"], s["t_len"]] + s["dst"]


# ----------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    slot = D // 2 + D // GROUP  # bytes of one slot of K (or V) of one head
    if op == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        n = case["M"] * (case["Hq"] + 2 * case["Hkv"]) * case["D"]
        return {"bytes": 2 * n * e + 4 * case["axes"] * case["M"], "flops": 10 * n}
    if op == "rows":
        n = case["layers"] * 2 * case["Hkv"] * case["rows"]
        return {"bytes": n * (2 * 2 * D + slot), "flops": 8 * n * D}
    if op == "attention":
        rows = case["N"] + 1
        keys = [T + rows for T in lengths(case)]
        b = sum(2 * case["Hkv"] * n * slot for n in keys) + 2 * 2 * case["B"] * rows * case["Hq"] * D
        f = sum(4 * D * case["Hq"] * rows * (n - rows + 1) for n in keys)
        return {"bytes": b, "flops": f}
    n = case["B"] * case["layers"] * 2 * case["Hkv"] * (case["N"] + 1)
    return {"bytes": n * (2 * 2 * D + slot) + case["B"] * (case["N"] + 1) * 16, "flops": 8 * n * D}


# ---------------------------------------------------------------------- exact

def _e4m3_grid():
    g = [m / 8 * 2.0 ** -6 for m in range(8)]
    g += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if not (e == 8 and m == 7)]
    return torch.tensor(g, dtype=torch.float64, device=DEV)


def _nearest(x, grid):
    """The member of an ascending grid nearest to each x >= 0; between two, the one of even index."""
    i = torch.searchsorted(grid, x.contiguous()).clamp(1, grid.numel() - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (x - lo > hi - x) | ((x - lo == hi - x) & (i % 2 == 0))
    return torch.where(up, hi, lo)


def _exact_values(x, g):
    """The values that a row's 4-bit form stands for, in 64 bits."""
    t = x.double() / float(torch.tensor(g, dtype=torch.float32))
    groups = t.reshape(*t.shape[:-1], -1, GROUP)
    s = _nearest(groups.abs().max(-1, keepdim=True).values / 6.0, _e4m3_grid())
    ok = s > 0
    q = _nearest(groups.abs() / torch.where(ok, s, torch.ones_like(s)), torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV))
    return (torch.sign(groups) * q * s * ok).reshape(t.shape) * float(torch.tensor(g, dtype=torch.float32))


def _exact_cache(c, name, h, n, g):
    """One head's cached values from the bits: (-1)^s (1 + f/2) 2^(e-1), f / 2 where e is 0."""
    b = c[name][h, :n].long()
    x = torch.empty(n, D, dtype=torch.float64, device=DEV)
    for odd in (0, 1):
        u = b >> 4 if odd else b & 15
        e, f = (u >> 1) & 3, (u & 1).double()
        m = torch.where(e > 0, (1 + f / 2) * torch.exp2(e.double() - 1), f / 2)
        x[:, odd::2] = torch.where(u > 7, -m, m)
    w = c[name + "_scale"][h, :n].long()
    e, f = (w >> 3) & 15, (w & 7).double()
    s = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 8 * 2.0 ** -6)
    return x * s.repeat_interleave(GROUP, 1) * float(torch.tensor(g, dtype=torch.float32))


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        M, Hq, Hkv, Dh, T = case["M"], case["Hq"], case["Hkv"], case["D"], case["T"]
        half = Dh // 2
        x = s["qkv"].double().reshape(M, -1, Dh)
        ax = frequency_axis(case)
        out = x.clone()
        for first, count, w in ((0, Hq, s["q_norm"]), (Hq, Hkv, s["k_norm"])):
            y = x[:, first:first + count]
            if w is not None:
                y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / Dh + 1e-6) * w.double()
            z = torch.complex(y[..., :half], y[..., half:])
            for j in range(half):
                a = s["pos"][ax[j]].double() * math.exp(-2 * j / Dh * math.log(case["theta"]))
                z[..., j] *= torch.polar(torch.ones_like(a), a).unsqueeze(1)
            out[:, first:first + count] = torch.cat((z.real, z.imag), -1)
        k, v = s["k"].double(), s["v"].double()
        k[:, T:T + M] = out[:, Hq:Hq + Hkv].transpose(0, 1)
        v[:, T:T + M] = out[:, Hq + Hkv:].transpose(0, 1)
        return [out[:, :Hq], k, v]
    if op == "rows":
        return torch.stack([torch.stack((_exact_values(x[0], s["k_global"]), _exact_values(x[1], s["v_global"])))
                            for x in s["src"]])
    if op == "attention":
        rows, G, out = case["N"] + 1, case["Hq"] // case["Hkv"], s["out"].double()
        for r, T in enumerate(lengths(case)):
            n, c = T + rows, s["caches"][r]
            hide = torch.zeros(rows, n, dtype=torch.float64, device=DEV)
            hide[:, T:][~s["trees"][r]["seen"]] = -math.inf
            for h in range(case["Hkv"]):
                k, v = _exact_cache(c, "k", h, n, s["k_global"]), _exact_cache(c, "v", h, n, s["v_global"])
                for i in range(h * G, h * G + G):
                    z = s["q"][r, :, i].double() @ k.t() / math.sqrt(D) + hide
                    w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
                    out[r, :, i] = w @ v
        return out
    B, L = case["B"], case["L"]
    a, tok, root, length, rest = [], [], [], [], []
    for r in range(B):
        t = s["trees"][r]
        parent, token, best = t["parent"].tolist(), t["token"].tolist(), s["argmax"][r].tolist()
        path = [0]
        while True:
            child = [i for i, p in enumerate(parent) if p == path[-1] and token[i] == best[path[-1]]]
            if not child:
                break
            path.append(child[0])
        x = s["src"][r]
        vals = torch.stack((_exact_values(x[:, 0], s["k_global"]), _exact_values(x[:, 1], s["v_global"])), 1)
        moved = vals.clone()
        moved[:, :, :, :len(path)] = vals[:, :, :, path]
        rest.append(moved)
        a.append(len(path) - 1)
        tok.append([token[i] for i in path[1:]] + [0] * (L - len(path) + 1))
        root.append(best[path[-1]])
        length.append(s["T"][r] + len(path))
    i32 = dict(dtype=torch.int32, device=DEV)
    return [torch.tensor(a, **i32), torch.tensor(tok, **i32), torch.tensor(root, **i32), torch.tensor(length, **i32)] + rest
