"""Refusals of the 4-bit calls at the ends of their arguments' ranges (CPU only)."""
import ctypes

import pytest

from _util import ensure_built
from test_kv4_abi import INVALID, ONE, UNSUPPORTED, tree, view


@pytest.fixture(scope="module")
def glib():
    ensure_built()
    import tree_verified_block_gb300 as g
    return g.lib()


def test_a_scale_that_overflows_with_a_cache_s_factor_is_refused(glib):
    import tree_verified_block_gb300._binding as b
    views = (b.KV4C * 2)(view(k_global=1.0), view(k_global=2.0 ** 60, t_len=128))
    trees = (b.TreeC * 2)(tree(), tree())

    def call(scale):
        # an out that overlaps q is refused after the scale: no launch either way
        return glib.glance_kv4_tree_attention(ONE, 4, ctypes.addressof(views), ctypes.addressof(trees), 2, scale, ONE, ONE, 1 << 30, None)
    assert call(2.0 ** 68) == INVALID and b"request 1" in glib.glance_last_error()
    assert call(2.0 ** 127.9) == INVALID and b"request 0" in glib.glance_last_error()
    assert call(2.0 ** 66) == INVALID and b"overlaps" in glib.glance_last_error()


def test_rows_calls_take_32767_layers_times_heads(glib):
    import tree_verified_block_gb300._binding as b
    layers = (b.KV4C * 128)(*[view(n_kv_heads=256) for _ in range(128)])
    p = ctypes.addressof(layers)
    assert glib.glance_kv4_write_rows(ONE, p, 128, 1, None) == UNSUPPORTED
    assert glib.glance_kv4_read_rows(p, 128, 0, 1, ONE, None) == UNSUPPORTED and b"32767" in glib.glance_last_error()
    # one layer fewer passes these checks: the next one that fails is the slots'
    assert glib.glance_kv4_read_rows(p, 127, 512, 1, ONE, None) == INVALID and b"t_cap" in glib.glance_last_error()
