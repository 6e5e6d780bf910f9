"""Sampling from rows of logits (glance_sample) against the oracle in 64 bits.

Tokens have to be the oracle's, also where two values are close (the kernel
compares those in 64 bits). Where a token's place at top_p's border is nearer to
it than weights are good to, 2^-21 of the sum (a weight to 2^-23 and its step's
rounding, sums in 64 bits), it is the oracle's draw with the border to either
side. The gap is the difference of two values that are good to 1e-9 each (pairs
of floats; logarithms to 1e-10, of -ln u relatively: over 0.35 at the least where
its series is longest), rounded to fp32."""
import numpy as np
import pytest
import torch

from oracle.truncated_sampling import kept_tokens, sample_row

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
NEAR = 2.0 ** -21


def draw(dev, logits, T=None, k=None, p=None, m=None, seed=5, pos=None, seq=None, gap=True):
    import tree_verified_block_gb300 as g
    M = logits.shape[0]
    t = lambda v, dt: None if v is None else torch.tensor(v, dtype=dt, device=dev)
    pos = torch.arange(100, 100 + M, dtype=torch.int32, device=dev) if pos is None else t(pos, torch.int32)
    tokens = torch.full((M,), -9, dtype=torch.int32, device=dev)
    gaps = torch.full((M,), -9.0, device=dev) if gap else None
    g.sample(logits, t(T, F32), t(k, torch.int32), t(p, F32), t(m, F32), seed, pos, t(seq, torch.int32), tokens, gaps)
    return tokens.cpu().numpy(), None if gaps is None else gaps.cpu().numpy().astype(np.float64), pos.cpu().numpy()


def check(dev, logits, T, k, p, m, seed=5, seq=None):
    M = logits.shape[0]
    tok, gap, pos = draw(dev, logits, T, k, p, m, seed, seq=seq)
    x = logits.double().cpu().numpy()
    for i in range(M):
        Ti = np.float32(T[i]) if T is not None else np.float32(1)
        at = lambda share: sample_row(x[i], seed, int(pos[i]), seq[i] if seq else 0, Ti, k[i] if k else 0, share, m[i] if m else 0.0)
        want, g64, near = at(p[i] if p else 1.0)
        if near < NEAR:
            assert tok[i] in [at(p[i] * f)[0] for f in (1 - NEAR, 1, 1 + NEAR)], (i, tok[i])
            continue
        assert tok[i] == want, (i, tok[i], want, g64, near)
        if np.isinf(g64):
            assert np.isinf(gap[i])
        else:
            assert abs(gap[i] - g64) <= 2.0 ** -23 * abs(g64) + 2e-9, (i, gap[i], g64)


def rows(dev, M, V, dtype, seed, std=2.0, peak=10.0, masked=0.0):
    gen = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(M, V, generator=gen, device=dev) * std
    n = min(V, 60)
    x[:, torch.randperm(V, generator=gen, device=dev)[:n]] += peak * torch.exp(-torch.arange(n, device=dev) / 9)
    if masked:
        stop = torch.rand(M, V, generator=gen, device=dev) < masked
        stop[:, V // 2] = False
        x.masked_fill_(stop, float("-inf"))
    return x.to(dtype)


CASES = [(0.7, 20, 0.8, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 0, 1.0, 0.0), (1.3, 0, 1.0, 0.05), (0.0, 5, 0.3, 0.1), (0.6, 1, 1.0, 0.0),
         (1.0, 50, 1.0, 0.0), (1.5, 1000, 0.9, 0.0), (2.0, 0, 0.999, 0.001), (0.05, 40, 0.9, 0.0), (1.0, 0, 0.0, 0.0), (1.0, 3, 0.5, 1.0),
         (3.0, 3000, 0.97, 0.0), (1.0, 10 ** 9, 2.0, -1.0)]


@pytest.mark.parametrize("V", [2, 3, 5, 64, 257, 1000, 4099, 32000, 151936])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_every_rule(dev, clean_status, V, dtype):
    for s, kw in enumerate((dict(), dict(std=1.0, peak=0.0), dict(masked=0.9))):
        x = rows(dev, len(CASES), V, dtype, V + s, **kw)
        T, k, p, m = (list(c) for c in zip(*CASES))
        check(dev, x, T, k, p, m, seed=V * 7 + (s << 40), seq=[i % 3 for i in range(len(CASES))])


def test_unaligned_and_strided_rows(dev, clean_status):
    for dtype in (F32, BF):
        for V, stride, off in ((1001, 1001, 1), (5000, 5003, 3), (40000, 40001, 0), (262144, 262147, 1)):
            M = 3
            flat = rows(dev, 1, off + M * stride, dtype, V).flatten()
            x = flat[off:].as_strided((M, V), (stride, 1), off)
            check(dev, x, [0.8] * M, [30] * M, [0.9] * M, None)
            check(dev, x, None, None, [0.97] * M, None)


@pytest.mark.parametrize("V", [3001, 151936])
def test_more_than_a_list_of_candidates(dev, clean_status, V):
    """Flat rows, rows of few distinct values and rows of one: the border lies among thousands of tokens or ties."""
    gen = torch.Generator(device=dev).manual_seed(V)
    flat = torch.rand(6, V, generator=gen, device=dev) * 0.01
    steps = torch.randint(0, 4, (6, V), generator=gen, device=dev).float() * 0.25
    one = torch.full((6, V), -3.5, device=dev)
    zero = torch.where(torch.rand(6, V, generator=gen, device=dev) < 0.5, 0.0, -0.0)  # equal: ties go by the id
    n = min(V, 100000)
    for x in (flat, steps, one, zero, flat.to(BF), steps.to(BF)):
        check(dev, x, [1.0, 1.0, 0.5, 4.0, 1.0, 1.0], [0, 2500, n // 2, 0, n // 2, n - 1], [0.5, 1.0, 1.0, 0.9999, 0.7, 0.999], None)


def test_top_p_under_a_wide_spread(dev, clean_status):
    """Weights over hundreds of nats, where all but the first few are outside the histogram."""
    x = -torch.arange(5000, dtype=F32, device=dev).flip(0)[None].repeat(5, 1) * 0.37
    x = x[:, torch.randperm(5000, generator=torch.Generator(device=dev).manual_seed(1), device=dev)]
    check(dev, x, [1.0, 0.1, 20.0, 100.0, 1.0], [0, 400, 4000, 0, 300], [0.99, 1.0, 0.9, 0.5, 0.999999], [0, 0, 0, 0, 1e-9])


def test_close_calls_are_decided_in_64_bits(dev, clean_status):
    """Two tokens whose perturbed values differ by less than fp32 resolves."""
    from oracle.sampling import gumbel_noise
    V, rows_ = 400, []
    for pos in range(100, 130):
        g = gumbel_noise(5, 0, pos, V)
        a, b = 17, 301
        x = np.full(V, -50.0, dtype=np.float32)
        x[a] = 1.0
        x[b] = np.float32(1.0 + g[a] - g[b])  # nearest: within 2^-24 of a tie
        rows_.append(x)
    x = torch.from_numpy(np.stack(rows_)).to(dev)
    check(dev, x, None, None, None, None)
    check(dev, x, None, [2] * 30, None, None)


def test_draws_have_the_kept_distribution(dev, clean_status):
    import tree_verified_block_gb300 as g
    n = 40000
    l = torch.tensor([2.0, 1.0, 1.5, -1.0, 0.5, float("-inf"), 2.0, 0.0], device=dev)
    full = lambda v, dt=F32: torch.full((n,), v, dtype=dt, device=dev)
    tokens = torch.zeros(n, dtype=torch.int32, device=dev)
    g.sample(l.expand(n, 8).contiguous(), full(1.3), full(5, torch.int32), full(0.9), None, 77, torch.arange(n, dtype=torch.int32, device=dev), None, tokens)
    mask, _ = kept_tokens(l.cpu().numpy(), 1.3, 5, 0.9)
    want = np.where(mask, np.exp(l.double().cpu().numpy() / 1.3), 0)
    want /= want.sum()
    got = np.bincount(tokens.cpu().numpy(), minlength=8) / n
    assert np.all(np.abs(got - want) <= 5 * np.sqrt(want * (1 - want) / n))  # five standard deviations


def test_with_nothing_cut_off_it_is_the_lm_head_s_draw(dev, clean_status):
    import tree_verified_block_gb300 as g
    M, d, V = 40, 128, 5000
    gen = torch.Generator(device=dev).manual_seed(8)
    h, W = torch.randn(M, d, generator=gen, device=dev), torch.randn(d, V, generator=gen, device=dev) * 0.3
    pos = torch.randint(0, 1 << 20, (M,), generator=gen, device=dev, dtype=torch.int32)
    seq = torch.randint(0, 9, (M,), generator=gen, device=dev, dtype=torch.int32)
    i32 = lambda: torch.zeros(M, dtype=torch.int32, device=dev)
    a, b, gap = i32(), i32(), torch.zeros(M, device=dev)
    g.lmhead_sample(h, W, 1 / 0.8, 1234567890123, pos, seq, a, gap, g.workspace(g.lmhead_argmax_workspace_bytes(M, d, V, F32), dev))
    g.sample((h.double() @ W.double()).float(), torch.full((M,), 0.8, device=dev), None, None, None, 1234567890123, pos, seq, b)
    sure = gap > 1e-3  # the LM head's fp32 sums of 128 products and this one's differ by rounding
    assert sure.sum() > 30 and torch.equal(a[sure], b[sure])


def test_bad_rows_are_refused_alone(dev):
    import tree_verified_block_gb300 as g
    for V in (100, 50000):
        x = torch.randn(9, V, device=dev)
        x[1, 5], x[2, V - 1], x[3] = float("nan"), float("inf"), float("-inf")
        st = torch.zeros(g.STATUS_WORDS, dtype=torch.int32, device=dev)
        for rows_, T, p, m, code in (([1, 2, 3], [1.0] * 9, [0.9] * 9, None, 1),
                                     ([1, 2, 3, 5, 6, 7, 8], [1, 1, 1, 1, 1, -1, float("nan"), float("inf"), 1e-40], None, None, None),
                                     ([1, 2, 3, 4, 6], [1.0] * 9, [1, 1, 1, 1, float("nan"), 1, 1, 1, 1], [0, 0, 0, 0, 0, 0, float("nan"), 0, 0], None)):
            g.reset_device_status()
            tok, gap, _ = draw(dev, x, T, None, p, m)
            g.get_status(st)
            assert st[0].item() in ((1,) if code else (1, 6)) and st[3] == st[0] and st[5] == 0
            bad = np.isin(np.arange(9), rows_)
            assert np.array_equal(tok == -1, bad) and np.array_equal(np.isnan(gap), bad) and np.all(tok[~bad] >= 0)
        g.reset_device_status()
        tok, _, _ = draw(dev, x[4:], [-2.0] * 5)
        g.get_status(st)
        assert st.tolist()[0] == 6 and np.all(tok == -1)
        g.reset_device_status()


def test_no_gap_captured_and_two_streams(dev, clean_status):
    import tree_verified_block_gb300 as g
    x = rows(dev, 20, 32000, BF, 3)
    tok, _, pos = draw(dev, x, [0.9] * 20, [0] * 20, [0.98] * 20, gap=False)
    T, p = torch.full((20,), 0.9, device=dev), torch.full((20,), 0.98, device=dev)
    pos = torch.from_numpy(pos).to(dev)
    outs, graphs, streams = [], [], [torch.cuda.Stream(dev) for _ in range(2)]
    for st in streams:
        out = torch.zeros(20, dtype=torch.int32, device=dev)
        st.wait_stream(torch.cuda.current_stream(dev))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            for _ in range(4):
                g.sample(x, T, None, p, None, 5, pos, None, out)
        outs.append(out)
        graphs.append(gr)
    torch.cuda.synchronize()
    for gr, st in zip(graphs, streams):
        with torch.cuda.stream(st):
            for _ in range(5):
                gr.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert np.array_equal(o.cpu().numpy(), tok)


@pytest.mark.parametrize("M", [1, 10, 19, 20, 300])
def test_row_counts_and_clustered_tokens(dev, clean_status, M):
    """Every cluster size; the likely tokens next to each other, so that one CTA has them all."""
    V = 40000
    gen = torch.Generator(device=dev).manual_seed(M)
    x = torch.randn(M, V, generator=gen, device=dev) - 4
    x[:, 300:2900] += 9
    pick = lambda *v: [v[i % len(v)] for i in range(M)]
    check(dev, x, pick(1.0, 0.6, 1.4), pick(1500, 0, 20, 1537), pick(0.9, 0.99, 1.0, 0.7, 0.95), pick(0.0, 0.01))
    check(dev, x.to(BF), pick(1.0, 1.4), pick(0, 1200), pick(0.97, 0.6, 0.999), None)


def test_the_same_row_gives_the_same_token_in_any_batch(dev, clean_status):
    import tree_verified_block_gb300 as g
    V = 50000
    x = rows(dev, 1, V, F32, 4)
    seen = []
    for M in (1, 19, 40, 200):
        t = lambda v, dt=F32: torch.full((M,), v, dtype=dt, device=dev)
        tokens, gap = t(0, torch.int32), t(0.0)
        g.sample(x.expand(M, V).contiguous(), t(1.1), t(0, torch.int32), t(0.98), None, 3, t(77, torch.int32), None, tokens, gap)
        seen += [tokens, gap]
    assert all(int(a) == int(seen[0][0]) for t in seen[::2] for a in t) and all(float(a) == float(seen[1][0]) for t in seen[1::2] for a in t)
