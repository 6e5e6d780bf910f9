"""Refusals of the 8-bit row, product and sampling calls: found on the host,
before any launch (CPU only), by the C ABI and by the binding."""
import ctypes

import pytest
import torch

from _util import ensure_built

INVALID, UNSUPPORTED = 1, 2
MB = 1 << 20
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def glib():
    ensure_built()
    import tree_verified_block_gb300 as g
    return g.lib()


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def rows(glib, **kw):
    a = dict(x=MB, xs=64, dtype=1, M=4, d=64, codes=2 * MB, cs=64, scales=3 * MB)
    a.update(kw)
    return glib.glance_q8_rows(vp(a["x"]), a["xs"], a["dtype"], a["M"], a["d"], vp(a["codes"]), a["cs"], vp(a["scales"]), None)


def norm(glib, **kw):
    a = dict(x=MB, xs=64, r=4 * MB, rs=64, dtype=1, M=4, d=64, w=5 * MB, eps=1e-6, t=6 * MB, ts=64, codes=2 * MB, cs=64, scales=3 * MB)
    a.update(kw)
    return glib.glance_q8_norm_rows(vp(a["x"]), a["xs"], vp(a["r"]), a["rs"], a["dtype"], a["M"], a["d"], vp(a["w"]), a["eps"],
                                    vp(a["t"]), a["ts"], vp(a["codes"]), a["cs"], vp(a["scales"]), None)


def read(glib, **kw):
    a = dict(codes=2 * MB, cs=64, scales=3 * MB, dtype=1, M=4, d=64, out=MB, os=64)
    a.update(kw)
    return glib.glance_q8_read_rows(vp(a["codes"]), a["cs"], vp(a["scales"]), a["dtype"], a["M"], a["d"], vp(a["out"]), a["os"], None)


BAD_ROWS = [(dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(dtype=2), INVALID), (dict(M=0), INVALID),
            (dict(M=-1), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(d=0), UNSUPPORTED), (dict(d=24, ), UNSUPPORTED),
            (dict(d=32784), UNSUPPORTED), (dict(d=16400, dtype=0), UNSUPPORTED), (dict(cs=48), INVALID), (dict(cs=72), INVALID),
            (dict(cs=1 << 41), INVALID), (dict(codes=2 * MB + 8), INVALID), (dict(scales=3 * MB + 2), INVALID),
            (dict(scales=2 * MB + 64), INVALID)]


@pytest.mark.parametrize("kw,status", BAD_ROWS)
def test_row_calls_refuse(glib, kw, status):
    assert rows(glib, **kw) == status and norm(glib, **kw) == status
    # reading takes scales anywhere, and rows as wide for either type
    if kw.get("scales") != 2 * MB + 64 and kw.get("d") != 16400:
        assert read(glib, **kw) == status
    assert glib.glance_last_error()


def test_row_calls_refuse_strides_alignment_and_overlaps(glib):
    for call in (rows, norm):
        for kw in (dict(x=None), dict(x=MB + 8), dict(xs=60), dict(xs=68), dict(xs=1 << 41), dict(codes=MB + 128), dict(scales=MB + 4),
                   dict(x=2 * MB - 512 + 16)):
            assert call(glib, **kw) == INVALID
    for kw in (dict(r=4 * MB + 8), dict(rs=60), dict(rs=68), dict(t=6 * MB + 4), dict(ts=32), dict(w=5 * MB + 4), dict(eps=-1.0),
               dict(eps=NAN), dict(eps=INF), dict(codes=4 * MB + 16), dict(codes=6 * MB + 16), dict(w=6 * MB + 16), dict(w=2 * MB),
               dict(t=MB + 128), dict(t=MB, ts=128), dict(t=4 * MB, ts=72), dict(t=4 * MB + 128)):
        assert norm(glib, **kw) == INVALID, kw
    for kw in (dict(out=None), dict(out=MB + 8), dict(os=60), dict(os=68), dict(out=2 * MB + 128), dict(out=3 * MB)):
        assert read(glib, **kw) == INVALID, kw


def linear(glib, **kw):
    a = dict(x=MB, xs=256, sx=2 * MB, M=4, w=3 * MB, ws=256, sw=4 * MB, N=64, K=256, gated=0, act=0, bias=None, r=None, rs=0, out=5 * MB,
             os=64, dtype=1)
    a.update(kw)
    return glib.glance_q8_linear(vp(a["x"]), a["xs"], vp(a["sx"]), a["M"], vp(a["w"]), a["ws"], vp(a["sw"]), a["N"], a["K"], a["gated"],
                                 a["act"], vp(a["bias"]), vp(a["r"]), a["rs"], vp(a["out"]), a["os"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INVALID), (dict(sx=None), INVALID), (dict(w=None), INVALID), (dict(sw=None), INVALID), (dict(out=None), INVALID),
    (dict(dtype=2), INVALID), (dict(act=4), INVALID), (dict(act=-1), INVALID), (dict(M=0), INVALID), (dict(M=(1 << 24) + 1), INVALID),
    (dict(N=0), UNSUPPORTED), (dict(N=60), UNSUPPORTED), (dict(N=(1 << 22) + 8), UNSUPPORTED), (dict(K=0), UNSUPPORTED),
    (dict(K=24), UNSUPPORTED), (dict(K=(1 << 20) + 16), UNSUPPORTED), (dict(xs=240), INVALID), (dict(xs=264), INVALID),
    (dict(ws=128), INVALID), (dict(ws=260), INVALID), (dict(os=56), INVALID), (dict(os=68), INVALID), (dict(xs=1 << 41), INVALID),
    (dict(r=6 * MB, rs=56), INVALID), (dict(r=6 * MB, rs=68), INVALID), (dict(r=6 * MB + 8, rs=64), INVALID),
    (dict(x=MB + 8), INVALID), (dict(w=3 * MB + 4), INVALID), (dict(out=5 * MB + 8), INVALID), (dict(sx=2 * MB + 2), INVALID),
    (dict(bias=6 * MB + 1), INVALID),
    (dict(out=MB + 512), INVALID), (dict(out=3 * MB + 64 * 256 - 16), INVALID), (dict(out=2 * MB), INVALID), (dict(out=4 * MB + 16), INVALID),
    (dict(out=5 * MB, bias=5 * MB + 16), INVALID), (dict(r=5 * MB + 128, rs=64), INVALID), (dict(r=5 * MB, rs=72), INVALID),
    # gated: twice the weights, scales and biases
    (dict(gated=1, out=3 * MB + 64 * 256), INVALID), (dict(gated=1, out=4 * MB + 4 * 64), INVALID)])
def test_linear_refuses(glib, kw, status):
    assert linear(glib, **kw) == status
    assert glib.glance_last_error()


def sample(glib, **kw):
    a = dict(logits=MB, stride=1000, dtype=0, M=4, V=1000, T=None, k=None, p=None, m=None, seed=1, pos=2 * MB, seq=None, tokens=3 * MB, gap=None)
    a.update(kw)
    return glib.glance_sample(vp(a["logits"]), a["stride"], a["dtype"], a["M"], a["V"], vp(a["T"]), vp(a["k"]), vp(a["p"]), vp(a["m"]),
                              a["seed"], vp(a["pos"]), vp(a["seq"]), vp(a["tokens"]), vp(a["gap"]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INVALID), (dict(pos=None), INVALID), (dict(tokens=None), INVALID), (dict(dtype=3), INVALID), (dict(M=0), INVALID),
    (dict(M=(1 << 20) + 1), INVALID), (dict(V=1), UNSUPPORTED), (dict(V=262145, stride=262145), UNSUPPORTED), (dict(stride=999), INVALID),
    (dict(stride=1 << 41), INVALID), (dict(logits=MB + 2), INVALID), (dict(logits=MB + 1, dtype=1), INVALID), (dict(T=4 * MB + 2), INVALID),
    (dict(tokens=3 * MB + 1), INVALID), (dict(tokens=MB + 4), INVALID), (dict(gap=MB + 8), INVALID), (dict(gap=3 * MB + 4), INVALID)])
def test_sample_refuses(glib, kw, status):
    assert sample(glib, **kw) == status
    assert glib.glance_last_error()


def test_binding_refuses_host_tensors_and_wrong_shapes():
    ensure_built()
    import tree_verified_block_gb300 as g
    f, c = torch.zeros(4, 64), torch.zeros(4, 64, dtype=torch.uint8)
    s, i = torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: g.q8_rows(f, c[:, :32], s), lambda: g.q8_rows(f, c.float(), s), lambda: g.q8_rows(f, c, s[:3]),
                 lambda: g.q8_rows(f.double(), c, s), lambda: g.q8_rows(f.t(), c.t(), s),
                 lambda: g.q8_norm_rows(f, f.to(torch.bfloat16), None, 1e-6, None, c, s),
                 lambda: g.q8_norm_rows(f, f[:3], None, 1e-6, None, c, s), lambda: g.q8_norm_rows(f, f, s, 1e-6, None, c, s),
                 lambda: g.q8_read_rows(c, s, f[:, :32]), lambda: g.q8_read_rows(c, s.int(), f),
                 lambda: g.q8_linear(c, s, c, s, f, act="relu"), lambda: g.q8_linear(c, s, c, s, torch.zeros(4, 8)),
                 lambda: g.q8_linear(c, s, c, s, torch.zeros(4, 4), gated=True),
                 lambda: g.q8_linear(c, s, c, s, torch.zeros(4, 4), bias=s[:2]),
                 lambda: g.q8_linear(c, s, c, s, torch.zeros(4, 4), residual=torch.zeros(4, 4, dtype=torch.bfloat16)),
                 lambda: g.sample(f, s[:2], None, None, None, 0, i, None, i), lambda: g.sample(f, None, s, None, None, 0, i, None, i),
                 lambda: g.sample(f, None, None, None, None, 0, None, None, i), lambda: g.sample(f.double(), None, None, None, None, 0, i, None, i),
                 # right in all but where they are
                 lambda: g.q8_rows(f, c, s), lambda: g.q8_read_rows(c, s, f), lambda: g.q8_linear(c, s, c, s, torch.zeros(4, 4)),
                 lambda: g.sample(f, None, None, None, None, 0, i, None, i)):
        with pytest.raises((ValueError, TypeError, RuntimeError, AssertionError)):
            call()
