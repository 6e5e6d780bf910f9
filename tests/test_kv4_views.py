"""Views of caches and trees as the 4-bit and rotary calls take them: what they
keep alive, what they pass on (CPU only)."""
import ctypes
import gc
import weakref

import pytest
import torch

from _util import ensure_built


@pytest.fixture(scope="module")
def b():
    ensure_built()
    import tree_verified_block_gb300._binding as b
    return b


class Array:
    """Stands for a tensor on device 0."""

    def __init__(self, shape=(1,), dtype=torch.uint8, contiguous=True):
        self.shape, self.dtype, self.contiguous, self.nbytes = torch.Size(shape), dtype, contiguous, 1 << 30

    def get_device(self):
        return 0

    def is_contiguous(self):
        return self.contiguous

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return 1 << 20


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


def test_views_do_not_change(b):
    """The C array is laid out once and holds addresses of the views' tensors."""
    layers = [view_of(b, b.KV4Layer) for _ in range(3)]
    v = b.Views(x for x in layers)
    assert list(v) == layers and v.n == len(v) == 3
    for change in (lambda: v.append(layers[0]), lambda: v.clear(), lambda: v.pop(), lambda: v.extend(layers), lambda: v.insert(0, 1),
                   lambda: v.__setitem__(0, layers[1]), lambda: v.__delitem__(0)):
        with pytest.raises(AttributeError):
            change()
    assert b._views(v, b.KV4Layer) is v
    twice = v
    twice += (layers[0],)  # a new tuple, which a call lays out anew
    assert v.n == len(v) == 3 and b._views(twice, b.KV4Layer).n == 4
    assert b._views(v[:2], b.KV4Layer).n == 2


def test_a_workspace_that_does_not_lie_in_one_piece_is_refused(b):
    """An expanded tensor of one byte says that it has any number of them."""
    layer, tree = view_of(b, b.KV4Layer), view_of(b, b.Tree)
    ws = Array(contiguous=False)
    q = Array((4, 4, 128), torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        b.kv4_tree_attention(q, layer, tree, 0.1, Array((4, 4, 128), torch.bfloat16), ws)
    i32 = [Array((4,), torch.int32) for _ in range(4)]
    with pytest.raises(ValueError, match="workspace"):
        b.kv4_accept_commit(tree, i32[0], layer, i32[1], i32[2], i32[3], ws)


def test_numbers_beyond_32_bits_are_refused(b):
    """2^32 + x reached the library as x: other rows, another plan."""
    layer = view_of(b, b.KV4Layer)
    for first in (2 ** 32, 2 ** 31, -2 ** 31 - 1):
        with pytest.raises(ValueError, match="first"):
            b.kv4_read_rows(layer, first, 16, Array((1, 2, 2, 16, 128), torch.bfloat16))
    with pytest.raises(ValueError, match="head_dim"):
        b.Rope(2 ** 32 + 128, 1e4, [64])
    with pytest.raises(ValueError, match="section"):
        b.Rope(128, 1e4, [2 ** 32 + 64])
    with pytest.raises(ValueError, match="rows"):
        b.kv4_tree_attention_workspace_bytes(2 ** 32 + 1, 4, layer)
    with pytest.raises(ValueError, match="n_layers"):
        b.kv4_accept_commit_workspace_bytes(1, 2 ** 32 + 1)
