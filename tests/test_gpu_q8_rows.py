"""Rows in 8 bits (glance_q8_norm_rows, glance_q8_rows, glance_q8_read_rows)
against the oracle in 64 bits.

Plain rows have to be equal. Normed rows: s is rounded as the oracle rounds it;
y = s w / sqrt(mean s^2 + eps) is off by the mean's sum (a thread adds at most 64
squares, 10 more levels join them, each step half of 2^-23, and half of that on
the root) and by root, quotient, mean and two products: under 45 * 2^-24 of y.
The value that a code stands for is then within half a step (2^-4 of y, or 2^-10
of the scale below the normal numbers) and that."""
import numpy as np
import pytest
import torch

from oracle import q8

pytestmark = pytest.mark.gpu

Y_ERR = 45 * 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.double().cpu().numpy()


def strided(M, d, pad, dtype, gen, dev, scale=1.0):
    return (torch.randn(M, d + pad, generator=gen, device=dev) * scale).to(dtype)[:, :d]


def empty8(M, d, pad, dev):
    return torch.full((M, d + pad), 0x55, dtype=torch.uint8, device=dev)


def check_values(y, values, scales):
    top = np.abs(y).max(axis=1)
    assert np.all(np.log2(scales) == np.round(np.log2(scales)))
    assert np.all(top <= 448 * scales * (1 + Y_ERR)) and np.all((top > 224 * scales * (1 - Y_ERR)) | (scales == 2.0 ** -126) | (top == 0))
    tol = np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10 * scales[:, None]) + Y_ERR * np.abs(y) * 1.1
    assert np.all(np.abs(values - y) <= tol), np.max(np.abs(values - y) - tol)


SHAPES = [(1, 16), (1, 4096), (3, 48), (5, 512), (7, 528), (130, 1024), (4, 4096), (9, 8192), (2, 12288), (1000, 64), (3, 16384)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", SHAPES + [(2, 32768)])
def test_plain_rows_are_the_oracle_s(dev, clean_status, dtype, M, d):
    import tree_verified_block_gb300 as g
    if dtype == F32 and d > 16384:
        pytest.skip("fp32 rows end at 16384")
    gen = torch.Generator(device=dev).manual_seed(M + d)
    x = strided(M, d, 16, dtype, gen, dev) * torch.exp2(torch.randint(-20, 20, (M, 1), generator=gen, device=dev)).to(dtype)
    wide = torch.zeros(M, d + 16, dtype=dtype, device=dev)
    wide[:, :d] = x
    x = wide[:, :d]
    x[0, d // 2:] *= 2.0 ** -12  # below the normal codes
    codes, scales = empty8(M, d, 32, dev), torch.zeros(M, device=dev)
    g.q8_rows(x, codes[:, :d], scales)
    want, scale = q8.quantise_rows(f64(x))
    assert np.array_equal(f64(scales), scale)
    assert np.array_equal(q8.code_values(codes[:, :d].cpu().numpy()) * scale[:, None], want)
    assert torch.all(codes[:, d:] == 0x55)
    for t in (BF, F32):
        out = torch.full((M, d + 8), 3.0, dtype=t, device=dev)
        g.q8_read_rows(codes[:, :d], scales, out[:, :d])
        assert np.array_equal(f64(out[:, :d]), want) and torch.all(out[:, d:] == 3)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,d", SHAPES)
@pytest.mark.parametrize("weight,residual,total", [(True, True, "new"), (True, True, "x"), (False, True, "residual"), (True, False, None)])
def test_normed_rows(dev, clean_status, dtype, M, d, weight, residual, total):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(3 * M + d)
    x, r = strided(M, d, 8, dtype, gen, dev, 3.0), strided(M, d, 24, dtype, gen, dev) if residual else None
    w = 1 + 0.5 * torch.randn(d, generator=gen, device=dev) if weight else None
    s = (x.float() + r.float()).to(dtype) if residual else x.clone()
    y = q8.norm_rows(f64(s), None if w is None else f64(w), 1e-5)
    t = {"new": torch.full((M, d + 16), 7.0, dtype=dtype, device=dev)[:, :d], "x": x, "residual": r, None: None}[total]
    codes, scales = empty8(M, d, 16, dev), torch.zeros(M, device=dev)
    g.q8_norm_rows(x, r, w, 1e-5, t, codes[:, :d].view(torch.float8_e4m3fn), scales)
    if t is not None:
        assert torch.equal(t, s)
    check_values(y, q8.code_values(codes[:, :d].cpu().numpy()) * f64(scales)[:, None], f64(scales))
    assert torch.all(codes[:, d:] == 0x55)
    if total == "new":
        assert torch.all(t._base[:, d:] == 7)


def test_rows_of_any_magnitude(dev, clean_status):
    """Squares that leave fp32's range, rows of zeros, rows that are tiny."""
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(5)
    for d in (128, 4096):
        x = torch.randn(7, d, generator=gen, device=dev)
        for i, f in enumerate((1.0, 2.0 ** 70, 2.0 ** 120, 2.0 ** -70, 2.0 ** -100, 0.0, 2.0 ** 64)):
            x[i] *= f
        codes, scales = empty8(7, d, 0, dev), torch.zeros(7, device=dev)
        for eps in (1e-6, 1e-30, 1e-36):
            g.q8_norm_rows(x, None, None, eps, None, codes, scales)
            check_values(q8.norm_rows(f64(x), None, float(np.float32(eps))), q8.code_values(codes.cpu().numpy()) * f64(scales)[:, None], f64(scales))
            assert torch.all(codes[5] & 127 == 0) and scales[5] == 1
        g.q8_rows(x, codes, scales)
        want, scale = q8.quantise_rows(f64(x))
        assert np.array_equal(f64(scales), scale) and np.array_equal(q8.code_values(codes.cpu().numpy()) * scale[:, None], want)


def test_a_row_that_is_not_finite_is_nan_alone(dev, clean_status):
    import tree_verified_block_gb300 as g
    for d, dtype in ((64, F32), (4096, BF)):
        x = torch.randn(6, d, device=dev).to(dtype)
        x[1, 3], x[2, d - 1], x[4, 0] = float("nan"), float("inf"), float("-inf")
        want = torch.tensor([False, True, True, False, True, False], device=dev)
        codes, scales, out = empty8(6, d, 0, dev), torch.zeros(6, device=dev), torch.zeros(6, d, device=dev)
        for norm in (False, True):
            if norm:
                g.q8_norm_rows(x, None, None, 1e-6, None, codes, scales)
            else:
                g.q8_rows(x, codes, scales)
            g.q8_read_rows(codes, scales, out)
            assert torch.equal(scales.isnan(), want) and torch.all(codes[want] == 0)
            assert torch.equal(out.isnan(), want[:, None].expand(6, d))


def test_rows_do_not_depend_on_their_place_nor_on_the_call(dev, clean_status):
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(9)
    x = torch.randn(300, 4096, generator=gen, device=dev).to(BF)
    codes, scales = empty8(300, 4096, 0, dev), torch.zeros(300, device=dev)
    g.q8_norm_rows(x, None, None, 1e-6, None, codes, scales)
    one, s1 = empty8(1, 4096, 0, dev), torch.zeros(1, device=dev)
    for i in (0, 17, 299):
        g.q8_norm_rows(x[i:i + 1], None, None, 1e-6, None, one, s1)
        assert torch.equal(one[0], codes[i]) and s1[0] == scales[i]


def test_captured_and_on_another_stream(dev, clean_status):
    import tree_verified_block_gb300 as g
    x, r = torch.randn(33, 512, device=dev).to(BF), torch.randn(33, 512, device=dev).to(BF)
    codes, scales, total = empty8(33, 512, 0, dev), torch.zeros(33, device=dev), torch.zeros_like(x)
    g.q8_norm_rows(x, r, None, 1e-6, total, codes, scales)
    want = codes.clone(), scales.clone(), total.clone()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        g.q8_norm_rows(x, r, None, 1e-6, total, codes, scales)
    for t in (codes, scales, total):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((codes, scales, total), want))
    codes.zero_()
    torch.cuda.synchronize()
    g.q8_norm_rows(x, r, None, 1e-6, total, codes, scales, stream=side)
    side.synchronize()
    assert torch.equal(codes, want[0])


def test_middles_of_normed_fp32_rows(dev, clean_status):
    """A value lands on the other side of the middle of two codes where y's error e, relative, reaches past it: one of
    2 e 2^3.5 values (middles are 2^-3 to 2^-4 of a value apart). What three products, root and quotient round (2^-24 in all)
    would make 16 of 2^24 values; with their remainders the sum of squares is left, whose first five levels 4 to 16 warps round
    by themselves (2^-25 each at most, 2^-27 in the mean, on the root half): 2 of 2^24. Up to 7 is within three times the root."""
    import tree_verified_block_gb300 as g
    gen = torch.Generator(device=dev).manual_seed(5)
    off = 0
    for M, d in ((2048, 2048), (1024, 4096), (4096, 1024), (512, 8192)):
        x, r = (torch.randn(M, d, generator=gen, device=dev) for _ in range(2))
        w = 1 + 0.3 * torch.randn(d, generator=gen, device=dev)
        codes, scales = empty8(M, d, 0, dev), torch.zeros(M, device=dev)
        g.q8_norm_rows(x, r, w, 1e-6, None, codes, scales)
        s = (x + r).double()
        y = s / torch.sqrt(s.pow(2).mean(1, keepdim=True) + float(np.float32(1e-6))) * w.double() / scales.double()[:, None]
        step = torch.exp2(torch.floor(torch.log2(y.abs())).clamp(min=-6) - 3)
        near = torch.round(y / step) * step  # to even where two are as near
        values = codes.view(torch.float8_e4m3fn).double()
        off += int((values != near)[y.abs() >= 2.0 ** -6].sum())
    assert off <= 7, off
