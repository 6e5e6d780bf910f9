"""Views of caches and trees as the 4-bit and rotary calls take them: what they
keep alive, what they pass on (CPU only)."""
import ctypes
import gc
import weakref

import pytest

from _util import ensure_built


@pytest.fixture(scope="module")
def b():
    ensure_built()
    import tree_verified_block_gb300._binding as b
    return b


class Array:
    """Stands for a device tensor."""

    def get_device(self):
        return 0


def view_of(b, kind):
    x = object.__new__(kind)
    if kind is b.Tree:
        x.anc, x.rows, x.L, x.c = Array(), 4, 2, b.TreeC(3, 2, 1)
    else:
        x.k, x.v, x.t_len = Array(), Array(), Array()
        x.c = (b.KV4C if kind is b.KV4Layer else b.KVC)(n_kv_heads=2, head_dim=128, t_cap=64)
    return x


@pytest.mark.parametrize("kind", ["Tree", "KVLayer", "KV4Layer"])
def test_a_view_that_a_call_took_alone_is_freed_with_its_last_reference(b, kind):
    kind = getattr(b, kind)
    was = gc.isenabled()
    gc.disable()  # the cyclic collector does not know what device memory waits for it
    try:
        x = view_of(b, kind)
        for _ in range(2):
            assert b._views(x, kind).n == 1
        kept = weakref.ref(x.anc if kind is b.Tree else x.k)
        del x
        assert kept() is None
    finally:
        if was:
            gc.enable()


@pytest.mark.parametrize("kind", ["KVLayer", "KV4Layer"])
def test_a_view_alone_is_passed_as_it_is_at_the_call(b, kind):
    kind = getattr(b, kind)
    x = view_of(b, kind)
    c = type(x.c)
    assert c.from_address(b._views(x, kind).at).t_cap == 64
    x.c.t_cap = 32
    assert c.from_address(b._views(x, kind).at).t_cap == 32
    x.c = c(n_kv_heads=2, head_dim=128, t_cap=16)
    assert c.from_address(b._views(x, kind).at).t_cap == 16
    assert ctypes.addressof(x.c) == b._views(x, kind).at
