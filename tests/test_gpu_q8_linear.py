"""Products of 8-bit rows (glance_q8_linear) against the oracle in 64 bits.

Products of codes are exact. The sum over K: K / 32 steps of the tensor core,
each adding to an fp32 accumulator a sum that it forms itself, and the partials
of at most 8 CTAs: (K / 16 + 16) steps of 2^-23, relative to the sum of the
magnitudes; two scales, the bias: 4 of 2^-24 of the magnitudes more. An
activation passes an error on with a slope of at most 1.13 (SiLU 1.10, GELU
1.13) and adds its own: e^x is good to 2 + 1.173 |x| steps of 2^-23, its
argument's rounding adds 4 |x| of 2^-24, the quotient 4 steps, erf 2 steps of
2^-23 times |v|. The gate's product and the residual's sum: one half step each;
the output's rounding: half a step."""
import numpy as np
import pytest
import torch

from oracle import q8

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ULP = 2.0 ** -23


def f64(t):
    return t.double().cpu().numpy()


def codes(rows, width, gen, dev, pad=0):
    x = torch.randn(rows, width + pad, generator=gen, device=dev)
    s = x.abs().amax(1) / 448
    return (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)[:, :width], s


def values(c, s):
    return q8.code_values(c.cpu().numpy()) * f64(s)[:, None]


def act_error(v, act):
    """The activation's own error, absolute."""
    a = np.abs(v)
    if act == "silu":
        return a * (2 + 1.173 * a + 2 * a + 4) * ULP
    if act == "gelu_tanh":
        z = 1.6 * (a + 0.045 * a ** 3)
        return np.minimum(a, np.abs(q8.activate(v, act)) * (2 + 1.173 * z + 4 * z + 4) * ULP + a * ULP)
    if act == "gelu":
        return 4 * a * ULP
    return 0.0


def check(dev, M, K, N, act="none", gated=False, bias=False, residual=False, out_dtype=F32, pads=(0, 0, 0, 0), in_place=False, seed=0):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(seed + 7 * M + K + N)
    rows = 2 * N if gated else N
    (x, xs), (w, ws) = codes(M, K, gen, dev, pads[0]), codes(rows, K, gen, dev, pads[1])
    ws = ws * 1.5 * K ** -0.5
    b = torch.randn(rows, generator=gen, device=dev) if bias else None
    r = torch.randn(M, N + pads[2], generator=gen, device=dev).to(out_dtype)[:, :N] if residual else None
    wide = torch.full((M, N + pads[3]), 9.0, dtype=out_dtype, device=dev)
    out = r if in_place else wide[:, :N]
    rr = None if r is None else f64(r)
    g.q8_linear(x, xs, w, ws, out, bias=b, act=act, gated=gated, residual=r)
    bb = None if b is None else f64(b)
    xv, wv = values(x, xs), values(w, ws)
    ref, _, size = q8.linear(xv, wv, bb, act, gated, rr)
    v = xv @ wv.T if bb is None else xv @ wv.T + bb
    ev = (K / 16 + 16 + 2) * ULP * size
    tol = 1.13 * ev[:, :N] + act_error(v[:, :N], act)
    if gated:
        a = q8.activate(v[:, :N], act)
        tol = tol * (np.abs(v[:, N:]) + ev[:, N:]) + np.abs(a) * ev[:, N:] + ULP / 2 * np.abs(a * v[:, N:])
    tol = (tol + ULP / 2 * np.abs(ref)) * 1.01 + (2.0 ** -8 if out_dtype == BF else 2.0 ** -24) * np.abs(ref)
    got = f64(out)
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()
    if not in_place:
        assert torch.all(wide[:, N:] == 9)


@pytest.mark.parametrize("M", [1, 2, 15, 16, 17, 31, 33, 64, 65, 100, 128, 129, 200, 256, 257, 300, 513])
def test_every_row_count(dev, clean_status, M):
    check(dev, M, 1024, 264)
    check(dev, M, 400, 200, act="silu", gated=True, out_dtype=BF)


@pytest.mark.parametrize("M", [3, 40, 128, 700])
@pytest.mark.parametrize("K,N", [(16, 8), (32, 128), (112, 136), (128, 256), (144, 8), (272, 248), (2064, 520), (4096, 64), (12288, 128)])
def test_odd_widths(dev, clean_status, M, K, N):
    check(dev, M, K, N, bias=True)


@pytest.mark.parametrize("M", [5, 64, 90, 600])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("out_dtype", [F32, BF])
def test_epilogues(dev, clean_status, M, act, gated, out_dtype):
    check(dev, M, 528, 328, act, gated, True, True, out_dtype)
    check(dev, M, 528, 328, act, gated, False, True, out_dtype, in_place=True)


@pytest.mark.parametrize("M", [1, 70, 300])
def test_strided(dev, clean_status, M):
    check(dev, M, 256, 152, "gelu", False, True, True, BF, pads=(16, 48, 8, 24))
    check(dev, M, 256, 152, "silu", True, False, True, F32, pads=(32, 16, 4, 12))


def test_projection_sizes(dev, clean_status):
    check(dev, 64, 4096, 4096, residual=True, out_dtype=BF)
    check(dev, 1, 4096, 6144, out_dtype=BF)
    check(dev, 33, 4096, 12288, act="silu", gated=True, out_dtype=BF)
    check(dev, 700, 4096, 2056, act="silu", gated=True, out_dtype=BF)


def test_scales_of_zero_and_large_sums(dev, clean_status):
    """Scales as checkpoints have them (no powers of two, zero); all codes at their largest."""
    import tree_verified_block_gb300 as g
    for M in (9, 300):
        x = torch.full((M, 4096), 0x7E, dtype=torch.uint8, device=dev)  # 448
        w = torch.full((64, 4096), 0x7E, dtype=torch.uint8, device=dev)
        w[1::2] = 0xFE
        xs, ws = torch.full((M,), 0.37, device=dev), torch.full((64,), 1e-3, device=dev)
        xs[2] = 0
        out = torch.zeros(M, 64, device=dev)
        g.q8_linear(x, xs, w, ws, out)
        want = np.outer(f64(xs), f64(ws)) * 4096 * 448.0 ** 2 * np.where(np.arange(64) % 2, -1, 1)
        assert np.all(np.abs(f64(out) - want) <= 300 * ULP * np.abs(want))


def test_a_nan_stays_in_its_row_or_column(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(2)
    for M in (20, 400):
        (x, xs), (w, ws) = codes(M, 512, gen, dev), codes(136, 512, gen, dev)
        x[3, 7], w[5, 100] = 0x7F, 0xFF
        xs[11], ws[70] = float("nan"), float("nan")
        out = torch.zeros(M, 136, device=dev)
        g.q8_linear(x, xs, w, ws, out)
        nan = torch.zeros(M, 136, dtype=torch.bool, device=dev)
        nan[[3, 11]] = True
        nan[:, [5, 70]] = True
        assert torch.equal(out.isnan(), nan)


def test_results_repeat(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(4)
    for M in (1, 64, 128, 1000):
        (x, xs), (w, ws) = codes(M, 2048, gen, dev), codes(1024, 2048, gen, dev)
        out = [torch.zeros(M, 1024, device=dev) for _ in range(2)]
        for o in out:
            for _ in range(3):
                g.q8_linear(x, xs, w, ws, o)
        assert torch.equal(out[0], out[1])


def test_captured_replayed_and_overlapping_calls(dev, clean_status):
    """Graphs of chained calls, and two streams at once: no call has memory of its own."""
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(6)
    sets = []
    for M in (64, 500):
        (x, xs), (w, ws) = codes(M, 1024, gen, dev), codes(1024, 1024, gen, dev)
        h, c, s, out = torch.zeros(M, 1024, dtype=BF, device=dev), torch.zeros_like(x), torch.zeros(M, device=dev), torch.zeros(M, 1024, device=dev)

        def chain(x=x, xs=xs, w=w, ws=ws, h=h, c=c, s=s, out=out):
            g.q8_linear(x, xs, w, ws, h, act="gelu")
            g.q8_rows(h, c, s)
            g.q8_linear(c, s, w, ws, out)
        chain()
        sets.append((chain, out, out.clone()))
    side = [torch.cuda.Stream(dev) for _ in sets]
    graphs = []
    for (chain, out, _), st in zip(sets, side):
        st.wait_stream(torch.cuda.current_stream(dev))
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            for _ in range(5):
                chain()
        graphs.append(gr)
        out.zero_()
    torch.cuda.synchronize()
    for gr, st in zip(graphs, side):
        with torch.cuda.stream(st):
            for _ in range(10):
                gr.replay()
    torch.cuda.synchronize()
    for _, out, want in sets:
        assert torch.equal(out, want)


def test_weights_written_just_before(dev, clean_status):
    """Weights may be read before the previous kernel has ended, but not before a row call has: nor through a product between."""
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(8)
    for M in (1, 64, 300):
        (x, xs), (w0, ws0) = codes(M, 4096, gen, dev), codes(2048, 4096, gen, dev)
        src = [torch.randn(2048, 4096, generator=gen, device=dev).to(BF) for _ in range(3)]
        w, ws = torch.zeros_like(w0), torch.zeros(2048, device=dev)
        want, other = [], torch.zeros(M, 2048, device=dev)
        for s in src:
            g.q8_rows(s, w, ws)
            torch.cuda.synchronize()
            want.append(torch.zeros(M, 2048, device=dev))
            g.q8_linear(x, xs, w, ws, want[-1])
            torch.cuda.synchronize()
        outs = [torch.zeros(M, 2048, device=dev) for _ in range(24)]
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            g.q8_rows(src[i % 3], w, ws)
            if i % 2:
                g.q8_linear(x, xs, w0, ws0, other)
            g.q8_linear(x, xs, w, ws, o)
        torch.cuda.synchronize()
        for i, o in enumerate(outs):
            assert torch.equal(o, want[i % 3]), (M, i)
