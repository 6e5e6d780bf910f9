"""glance_qk_norm_rope against the oracle in 64 bits."""
import numpy as np
import pytest
import torch

import workloads as W
from oracle import rope as orope

pytestmark = pytest.mark.gpu


def run(dev, B, M, Hq, Hkv, D, dtype, axes, sec, il, T, norm, theta=1e6, pos=None, gap=0, seed=0, eps=1e-6):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(seed + M * 7 + D)
    width = (Hq + 2 * Hkv) * D
    big = torch.randn(B * M, width + gap, generator=gen, device=dev).mul_(1.7).to(dtype)
    qkv = big[:, :width]
    qw = (1 + 0.3 * torch.randn(D, generator=gen, device=dev)) if norm & 1 else None
    kw = (1 + 0.3 * torch.randn(D, generator=gen, device=dev)) if norm & 2 else None
    if pos is None:
        pos = torch.randint(-50, 200000, (axes, B * M), generator=gen, device=dev, dtype=torch.int32)
    caches, t_lens = [], []
    for r in range(B):
        t_lens.append(torch.tensor([T + 3 * r], dtype=torch.int32, device=dev))
        caches.append([torch.full((Hkv, T + 3 * r + M + 5, D + 16), 9.0, dtype=dtype, device=dev)[:, :, :D] for _ in range(2)])
    views = [g.KVLayer(k, v, t) for (k, v), t in zip(caches, t_lens)]
    q_out = torch.full((B * M, Hq, D), 5.0, dtype=dtype, device=dev)
    g.qk_norm_rope(qkv, Hq, qw, kw, eps, pos, g.Rope(D, theta, sec, il), q_out, views if B > 1 else views[0])
    x = qkv.double().cpu().numpy().reshape(B * M, -1, D)
    p = pos.cpu().numpy()
    half_step = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24

    def want(y, w):
        w = None if w is None else w.double().cpu().numpy()
        o = orope.qk_norm_rope(y, w, p, theta, sec, il, eps)
        # fp32 arithmetic on the pair: the mean of D squares (log2 D + 3 rounded
        # steps), root, two products with w, sine and cosine (2^-22 absolute:
        # the angle to 2^-25 of half a turn, and their own rounding), two
        # products and a sum: under 32 steps of 2^-24 of |a| + |b|
        n = np.abs(orope.qk_norm_rope(y, w, np.zeros_like(p), theta, sec, il, eps))
        n = n + np.roll(n, D // 2, -1)
        return o, half_step * np.abs(o) + 32 * 2.0 ** -24 * n

    o, tol = want(x[:, :Hq], qw)
    assert np.all(np.abs(q_out.double().cpu().numpy() - o) <= tol)
    o, tol = want(x[:, Hq:Hq + Hkv], kw)
    for r in range(B):
        t0 = T + 3 * r
        k, v = (c.double().cpu().numpy() for c in caches[r])
        at = slice(r * M, r * M + M)
        assert np.all(np.abs(k[:, t0:t0 + M].transpose(1, 0, 2) - o[at]) <= tol[at])
        assert np.array_equal(v[:, t0:t0 + M].transpose(1, 0, 2), x[at, Hq + Hkv:])
        for c in (k, v):
            assert np.all(c[:, :t0] == 9) and np.all(c[:, t0 + M:] == 9)
        assert int(t_lens[r]) == t0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,Hq,Hkv,D,axes,sec,il,T,norm", [
    (1, 32, 8, 128, 1, None, False, 0, 3), (64, 32, 8, 128, 1, None, False, 700, 3), (37, 4, 2, 32, 1, None, False, 0, 0),
    (5, 8, 8, 64, 2, [20, 12], False, 3, 1), (9, 3, 1, 128, 3, [24, 20, 20], True, 11, 2),
    (2500, 8, 2, 128, 3, [24, 20, 20], True, 0, 3), (2433, 5, 1, 64, 4, [8, 8, 8, 8], True, 2, 3)])
def test_rows_match_the_formula(dev, clean_status, dtype, M, Hq, Hkv, D, axes, sec, il, T, norm):
    run(dev, 1, M, Hq, Hkv, D, dtype, axes, sec, il, T, norm)


def test_batch_strided_rows_and_far_positions(dev, clean_status):
    run(dev, 5, 33, 8, 2, 128, torch.bfloat16, 1, None, False, 7, 3, gap=24)
    run(dev, 16, 3, 4, 4, 64, torch.float32, 2, [16, 16], True, 0, 3, gap=8)
    far = torch.tensor([[2 ** 31 - 1, -2 ** 31, 10 ** 9 + 7, 0, 1, -1]], dtype=torch.int32, device=dev)
    # float64 angles of the oracle are off by 2^-53 * 2^31 = 2^-22 here, within the sine's share of the tolerance
    run(dev, 1, 6, 4, 2, 128, torch.float32, 1, None, False, 0, 0, pos=far)


def test_zero_rows_stay_zero_and_not_finite_rows_stay_alone(dev, clean_status):
    import tree_verified_block_gb300 as g
    qkv = torch.randn(4, 6 * 64, device=dev)
    qkv[1] = 0
    qkv[2, 5] = float("nan")
    qkv[3, 64] = float("inf")
    k, v = torch.zeros(2, 8, 64, device=dev), torch.zeros(2, 8, 64, device=dev)
    kv = g.KVLayer(k, v, torch.zeros(1, dtype=torch.int32, device=dev))
    w = torch.ones(64, device=dev)
    q = torch.empty(4, 2, 64, device=dev)
    g.qk_norm_rope(qkv, 2, w, w, 1e-6, torch.arange(4, dtype=torch.int32, device=dev)[None], g.Rope(64, 1e4), q, kv)
    assert torch.all(q[1] == 0) and torch.all(k[:, 1] == 0)
    assert q[2, 0].isnan().all() and q[2, 1].isfinite().all() and q[0].isfinite().all()
    assert q[3, 0].isfinite().all() and q[3, 1].isnan().any() and k.isfinite().all()


def test_no_room_sets_status_2_and_leaves_the_cache(dev):
    import tree_verified_block_gb300 as g
    g.reset_device_status()
    k, v = torch.zeros(2, 8, 64, device=dev), torch.zeros(2, 8, 64, device=dev)
    kv = g.KVLayer(k, v, torch.full((1,), 5, dtype=torch.int32, device=dev))
    q = torch.zeros(4, 2, 64, device=dev)
    g.qk_norm_rope(torch.ones(4, 6 * 64, device=dev), 2, None, None, 1e-6, torch.zeros(1, 4, dtype=torch.int32, device=dev),
                   g.Rope(64, 1e4), q, kv)
    st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
    g.get_status(st)
    assert st.tolist() == [2, 0, 0, 0, 0, 2]  # reported with the dense layers
    g.reset_device_status()
    assert torch.all(k == 0) and torch.all(v == 0)


def test_the_layers_projection_and_this_call_agree(dev, clean_status):
    """glance_dense_qkv rotates and norms as this call does on its own product."""
    import tree_verified_block_gb300 as g
    M, d, Hq, Hkv = 32, 256, 4, 2
    gen = torch.Generator(device=dev).manual_seed(3)
    h = torch.randn(M, d, generator=gen, device=dev).to(torch.bfloat16)
    Wq = (torch.randn(d, (Hq + 2 * Hkv) * 128, generator=gen, device=dev) * 0.06).to(torch.bfloat16)
    w = 1 + 0.2 * torch.randn(128, generator=gen, device=dev)
    pos = torch.randint(0, 3000, (M,), generator=gen, device=dev, dtype=torch.int32)
    z = lambda: [torch.zeros(Hkv, 64, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    t = torch.zeros(1, dtype=torch.int32, device=dev)
    (k0, v0), (k1, v1) = z(), z()
    q0, q1 = (torch.empty(M, Hq, 128, dtype=torch.bfloat16, device=dev) for _ in range(2))
    g.dense_qkv(h, Wq, Hq, None, w, w, 1e-6, pos, 1e6, q0, g.KVLayer(k0, v0, t))
    prod = (h.double() @ Wq.double()).to(torch.bfloat16)
    g.qk_norm_rope(prod, Hq, w, w, 1e-6, pos[None], g.Rope(128, 1e6), q1, g.KVLayer(k1, v1, t))
    # the product is rounded to bf16 in between (2^-8 of each element; the norm
    # passes that on, the rotation mixes two) and both results are (2^-8 each)
    for a, b in ((q0, q1), (k0, k1), (v0, v1)):
        a, b = a.float(), b.float()
        assert torch.all((a - b).abs() <= 2 ** -8 * (2 * b.abs() + 4 * b.abs().amax(-1, keepdim=True)))
