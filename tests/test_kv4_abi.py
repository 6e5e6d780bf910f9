"""Refusals of the 4-bit cache and rotary calls: found on the host, before any
launch (CPU only), by the C ABI and by the binding."""
import ctypes

import pytest
import torch

from _util import ensure_built

INVALID, UNSUPPORTED, CAPACITY = 1, 2, 3
ONE = ctypes.c_void_p(4096)


@pytest.fixture(scope="module")
def glib():
    ensure_built()
    import tree_verified_block_gb300 as g
    return g.lib()


def view(**kw):
    import tree_verified_block_gb300._binding as b
    a = dict(k=1 << 20, k_scale=1 << 21, v=1 << 22, v_scale=1 << 23, k_global=1.0, v_global=0.5, n_kv_heads=2,
             head_dim=128, t_cap=512, head_stride=512, t_len=64)
    a.update(kw)
    return b.KV4C(*[a[n] for n, _ in b.KV4C._fields_])


def tree(n=15, L=7, **kw):
    import tree_verified_block_gb300._binding as b
    t = b.TreeC(n, L, (n + 64) // 64, 16, 16, 16, 16, 16, 16)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


BAD_VIEWS = [(dict(k=None), INVALID), (dict(v_scale=None), INVALID), (dict(t_len=None), INVALID),
             (dict(k=(1 << 20) + 8), INVALID), (dict(k_scale=(1 << 21) + 8), INVALID),
             (dict(head_dim=64), UNSUPPORTED), (dict(head_stride=510), INVALID), (dict(t_cap=511, head_stride=511), INVALID),
             (dict(n_kv_heads=0), INVALID), (dict(t_cap=8), INVALID), (dict(k_global=0.0), INVALID),
             (dict(k_global=float("nan")), INVALID), (dict(v_global=float("inf")), INVALID), (dict(v_global=-1.0), INVALID),
             (dict(t_cap=(1 << 30) + 2, head_stride=(1 << 30) + 2), UNSUPPORTED)]


@pytest.mark.parametrize("kw,status", BAD_VIEWS)
def test_bad_views_are_refused_by_every_call(glib, kw, status):
    x, t = view(**kw), tree()
    p = ctypes.addressof(x)
    assert glib.glance_kv4_write_rows(ONE, p, 1, 16, None) == status
    assert glib.glance_kv4_read_rows(p, 1, 0, 16, ONE, None) == status
    assert glib.glance_kv4_tree_attention(ONE, 4, p, ctypes.addressof(t), 1, 0.1, ctypes.c_void_p(1 << 24), ONE, 1 << 30,
                                          None) == status
    assert glib.glance_kv4_accept_commit(ctypes.addressof(t), 1, ONE, None, 0.0, p, 1, ONE, ONE, ONE, None, ONE, 256,
                                         None) == status
    assert glib.glance_last_error()


def test_rows_calls_refuse(glib):
    x = view()
    p = ctypes.addressof(x)
    for n_layers, rows in ((0, 1), (129, 1), (1, 0), (1, 513)):
        assert glib.glance_kv4_write_rows(ONE, p, n_layers, rows, None) == INVALID
        assert glib.glance_kv4_read_rows(p, n_layers, 0, rows, ONE, None) == INVALID
    assert glib.glance_kv4_write_rows(None, p, 1, 1, None) == INVALID
    assert glib.glance_kv4_write_rows(ctypes.c_void_p(4096 + 16), p, 1, 1, None) == INVALID
    assert glib.glance_kv4_read_rows(p, 1, -1, 1, ONE, None) == INVALID
    assert glib.glance_kv4_read_rows(p, 1, 500, 13, ONE, None) == INVALID
    assert glib.glance_kv4_read_rows(p, 1, 2 ** 31 - 1, 12, ONE, None) == INVALID
    import tree_verified_block_gb300._binding as b
    two = (b.KV4C * 2)(view(), view(k_global=2.0))
    assert glib.glance_kv4_write_rows(ONE, ctypes.addressof(two), 2, 1, None) == INVALID
    assert b"same t_len, geometry and globals" in glib.glance_last_error()


def test_attention_refuses(glib):
    x = view()
    p = ctypes.addressof(x)

    def call(t, B=1, Hq=4, scale=0.1, q=4096, out=1 << 24, ws=4096, n=1 << 30):
        return glib.glance_kv4_tree_attention(ctypes.c_void_p(q), Hq, p, ctypes.addressof(t), B, scale, ctypes.c_void_p(out),
                                              ctypes.c_void_p(ws), n, None)
    assert call(tree(n=256, mask_words=5)) == INVALID
    assert call(tree(n=-1, mask_words=0)) == INVALID
    assert call(tree(mask_words=2)) == INVALID
    assert call(tree(anc=None)) == INVALID
    assert call(tree(), B=0) == INVALID and call(tree(), B=17) == INVALID
    assert call(tree(), Hq=3) == INVALID and call(tree(), Hq=0) == INVALID
    assert call(tree(), Hq=6) == UNSUPPORTED and call(tree(), Hq=32) == UNSUPPORTED
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(tree(), scale=s) == INVALID
    assert call(tree(), q=4104) == INVALID and call(tree(), out=(1 << 24) + 2) == INVALID
    assert call(tree(), out=4096 + 256) == INVALID  # overlaps q
    assert call(tree(), n=16) == CAPACITY and call(tree(), ws=None) == CAPACITY
    assert call(tree(), ws=4096 + 16) == INVALID
    t = tree()
    assert glib.glance_kv4_tree_attention(None, 4, p, ctypes.addressof(t), 1, 0.1, ONE, ONE, 1 << 30, None) == INVALID
    size = glib.glance_kv4_tree_attention_workspace_bytes
    assert size(1, 64, 4, p) >= 256 and size(1, 1, 4, p) >= 256
    assert size(0, 64, 4, p) == 0 and size(17, 64, 4, p) == 0 and size(1, 257, 4, p) == 0 and size(1, 0, 4, p) == 0
    assert size(1, 64, 3, p) == 0 and size(1, 64, 0, p) == 0 and size(1, 64, 4, None) == 0


def test_commit_refuses(glib):
    import tree_verified_block_gb300._binding as b
    x = (b.KV4C * 2)(view(), view(t_cap=256))

    def call(t=None, B=1, n_layers=1, gap=None, gated=None, ws=4096, n=256, arr=x):
        t = t or tree()
        ts = (b.TreeC * 2)(t, t)
        return glib.glance_kv4_accept_commit(ctypes.addressof(ts), B, ONE, gap, 0.5, ctypes.addressof(arr), n_layers, ONE,
                                             ONE, ONE, gated, ctypes.c_void_p(ws), n, None)
    assert call(n_layers=2) == INVALID and b"share geometry" in glib.glance_last_error()
    assert call(B=0) == INVALID and call(B=17) == INVALID and call(n_layers=0) == INVALID and call(n_layers=129) == INVALID
    assert call(B=2) == INVALID and b"share t_len" in glib.glance_last_error()
    assert call(gap=ONE) == INVALID and call(gated=ONE) == INVALID
    assert call(ws=None) == INVALID and call(n=8) == CAPACITY and call(ws=4097) == INVALID
    assert call(tree(n=0, mask_words=1)) == INVALID and call(tree(L=17)) == INVALID and call(tree(parent=None)) == INVALID
    assert glib.glance_kv4_accept_commit_workspace_bytes(16, 60) == 256
    assert glib.glance_kv4_accept_commit_workspace_bytes(16, 61) == 0
    assert glib.glance_kv4_accept_commit_workspace_bytes(1, 129) == 0


def test_rope_init(glib):
    import tree_verified_block_gb300 as g
    r = g.Rope(128, 1e6, [24, 20, 20], True)
    assert list(r.c.axis)[:7] == [0, 1, 2, 0, 1, 2, 0] and list(r.c.axis)[60:] == [0, 0, 0, 0]
    for j in (0, 1, 31, 63):  # turns of 2^64
        want = 1e6 ** (-2 * j / 128) / (2 * 3.141592653589793) * 2.0 ** 64
        assert abs(r.c.turn[j] - want) <= 2.0 ** -52 * want * 4 + 0.5  # a whole number
    assert g.Rope(64, 1e4, [16, 16]).c.axis[15] == 0 and g.Rope(64, 1e4, [16, 16]).c.axis[16] == 1
    bad = [dict(head_dim=96, theta=1e4), dict(head_dim=128, theta=0.0), dict(head_dim=128, theta=float("inf")),
           dict(head_dim=128, theta=-2.0), dict(head_dim=128, theta=1e4, sections=[32, 31]),
           dict(head_dim=128, theta=1e4, sections=[64, 0]), dict(head_dim=128, theta=1e4, sections=[65, -1]),
           dict(head_dim=128, theta=1e4, sections=[10] * 5), dict(head_dim=32, theta=1e4, sections=[2, 12, 2], interleaved=True)]
    for kw in bad:
        with pytest.raises(g.GlanceError):
            g.Rope(**kw)


def test_rope_call_refuses(glib):
    import tree_verified_block_gb300 as g
    import tree_verified_block_gb300._binding as b
    r = g.Rope(128, 1e4)
    kv = b.KVC(1 << 30, 1 << 31, 1, 2, 128, 64, 64 * 128, 128, 64)

    def call(qkv=1 << 20, dtype=1, B=1, M=16, stride=1024, Hq=4, eps=1e-6, pos=4096, rope=r.c, q_out=1 << 24, kvs=kv):
        return glib.glance_qk_norm_rope(ctypes.c_void_p(qkv), dtype, B, M, stride, Hq, None, None, eps, ctypes.c_void_p(pos),
                                        ctypes.addressof(rope), ctypes.c_void_p(q_out), ctypes.addressof(kvs), None)
    assert call(qkv=None) == INVALID and call(pos=None) == INVALID and call(q_out=None) == INVALID
    assert call(dtype=2) == INVALID and call(B=0) == INVALID and call(B=17) == INVALID and call(M=0) == INVALID
    assert call(M=65) == INVALID and call(stride=1016) == INVALID and call(stride=1028) == INVALID and call(Hq=0) == INVALID
    assert call(eps=-1.0) == INVALID and call(eps=float("nan")) == INVALID
    assert call(qkv=(1 << 20) + 8) == INVALID and call(q_out=(1 << 24) + 4) == INVALID
    assert call(q_out=(1 << 20) + 1024) == INVALID and b"overlaps" in glib.glance_last_error()
    assert call(rope=b.RopeC()) == INVALID
    assert call(dtype=0) == INVALID  # the cache is bf16
    assert call(kvs=b.KVC(1 << 30, 1 << 31, 1, 2, 64, 64, 64 * 64, 64, 64)) == INVALID
    assert call(kvs=b.KVC(1 << 30, None, 1, 2, 128, 64, 64 * 128, 128, 64)) == INVALID
    assert call(kvs=b.KVC(1 << 30, 1 << 31, 1, 2, 128, 64, 63 * 128, 128, 64)) == INVALID
    assert call(kvs=b.KVC(1 << 30, 1 << 31, 1, 2, 128, 64, 64 * 129, 129, 64)) == INVALID
    two = (b.KVC * 2)(kv, kv)
    assert call(B=2, M=8, kvs=two) == INVALID and b"share a cache" in glib.glance_last_error()


def test_the_binding_refuses_host_tensors_and_wrong_shapes(glib):
    import tree_verified_block_gb300 as g
    z = torch.zeros((2, 16, 64), dtype=torch.uint8)
    s = torch.zeros((2, 16, 8), dtype=torch.uint8)
    t = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        g.KV4Layer(z, s, z, s, t)            # host memory
    with pytest.raises(ValueError):
        g.KV4Layer(z, s[:, :, :4], z, s, t)  # 8 scales a row
    with pytest.raises(ValueError):
        g.KV4Layer(z, s, z, s, t.long())
    with pytest.raises(ValueError):
        g.KV4Layer(z[:, ::2], s[:, ::2], z[:, ::2], s[:, ::2], t)  # rows not next to each other
    with pytest.raises(ValueError):
        g.KV4Layer(z[:1, :15], s[:1, :15], z[:1, :15], s[:1, :15], t)  # an odd number of slots
    with pytest.raises(ValueError):
        g.Views([])
    with pytest.raises(TypeError):
        g._binding._views(g.Views([type("X", (), {"c": t_c()})()]), g.KV4Layer)


def test_a_theta_without_finite_frequencies_is_refused(glib):
    import tree_verified_block_gb300 as g
    for theta in (5e-324, 1e-320):
        with pytest.raises(g.GlanceError):
            g.Rope(128, theta)
    assert g.Rope(128, 1e-300).c.turn[0] == g.Rope(128, 1e4).c.turn[0]  # frequency 0 is 1 for every theta


def test_views_are_of_one_kind_and_one_device(glib):
    import tree_verified_block_gb300._binding as b

    class Where:
        def __init__(self, dev):
            self.dev = dev

        def get_device(self):
            return self.dev

    def layer(*devs):
        x = object.__new__(b.KV4Layer)
        x.k, x.v, x.t_len = map(Where, devs)
        x.c = view()
        return x
    tree = object.__new__(b.Tree)
    tree.anc, tree.c = Where(0), b.TreeC()
    assert b.Views([layer(0, 0, 0), layer(0, 0, 0)]).dev == 0
    for bad in ([layer(0, 0, 1)], [layer(0, 0, 0), layer(1, 1, 1)]):
        with pytest.raises(ValueError):
            b.Views(bad)
    with pytest.raises(TypeError):
        b.Views([layer(0, 0, 0), tree])


def test_attention_workspace_refuses_more_heads_than_the_call(glib):
    x = view(n_kv_heads=1025)
    assert glib.glance_kv4_tree_attention_workspace_bytes(1, 1, 1025, ctypes.byref(x)) == 0


def t_c():
    import tree_verified_block_gb300._binding as b
    return b.TreeC()
