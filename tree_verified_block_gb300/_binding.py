"""ctypes binding of libglance.so: argument marshalling only.

Every step runs in the library's CUDA kernels. PyTorch provides device memory
and streams; tensors are passed as raw pointers. There is no fallback: if the
library is not built, every call raises.
"""
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libglance.so")

F32, BF16 = 0, 1
STATUS = {0: "GLANCE_OK", 1: "GLANCE_ERR_INVALID_ARG", 2: "GLANCE_ERR_UNSUPPORTED",
          3: "GLANCE_ERR_CAPACITY", 4: "GLANCE_ERR_CUDA", 5: "GLANCE_ERR_DEVICE"}
DEV_STATUS = {0: "ok", 1: "non-finite draft logits", 2: "tree does not fit the cache",
              3: "inconsistent tree", 4: "pipeline wait timed out",
              5: "index out of bounds (bounds-checked build)",
              6: "sampling parameters out of range"}

EXPORTS = [
    "glance_build_tree_workspace_bytes", "glance_build_tree",
    "glance_tree_attention_workspace_bytes", "glance_tree_attention",
    "glance_tree_attention_timeout_check",
    "glance_lmhead_argmax_workspace_bytes", "glance_lmhead_argmax", "glance_lmhead_argmax_noalloc",
    "glance_lmhead_packed_w_bytes", "glance_lmhead_pack_w", "glance_lmhead_argmax_packed",
    "glance_accept_commit_workspace_bytes", "glance_accept_commit",
    "glance_build_tree_batched_workspace_bytes", "glance_build_tree_batched",
    "glance_tree_attention_batched_workspace_bytes", "glance_tree_attention_batched",
    "glance_accept_commit_batched_workspace_bytes", "glance_accept_commit_batched",
    "glance_lmhead_argmax_entropy", "glance_lmhead_sample", "glance_accept_commit_gated",
    "glance_build_tree_shared_workspace_bytes", "glance_build_tree_shared",
    "glance_row_sumsq", "glance_dense_qkv",
    "glance_dense_residual", "glance_dense_swiglu",
    "glance_accept_commit_gated_batched",
    "glance_rope_init", "glance_qk_norm_rope",
    "glance_kv4_write_rows", "glance_kv4_read_rows",
    "glance_kv4_tree_attention_workspace_bytes", "glance_kv4_tree_attention",
    "glance_kv4_accept_commit_workspace_bytes", "glance_kv4_accept_commit",
    "glance_q8_rows", "glance_q8_norm_rows", "glance_q8_read_rows", "glance_q8_linear", "glance_sample",
    "glance_last_error", "glance_status_string", "glance_device_status",
    "glance_reset_device_status", "glance_get_status", "glance_kv_write_rows", "glance_clear_status", "glance_version",
]


class GlanceError(RuntimeError):
    def __init__(self, status, message):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class TreeC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("L", ctypes.c_int32), ("mask_words", ctypes.c_int32),
                ("token", ctypes.c_void_p), ("parent", ctypes.c_void_p),
                ("depth", ctypes.c_void_p), ("pos_id", ctypes.c_void_p),
                ("score", ctypes.c_void_p), ("anc", ctypes.c_void_p)]


class KVC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("t_cap", ctypes.c_int32), ("head_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("t_len", ctypes.c_void_p)]


class KV4C(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("k_global", ctypes.c_float), ("v_global", ctypes.c_float),
                ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("t_cap", ctypes.c_int32),
                ("head_stride", ctypes.c_int64), ("t_len", ctypes.c_void_p)]


class RopeC(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("turn", ctypes.c_uint64 * 64),
                ("axis", ctypes.c_uint8 * 64)]


_lib = None


def lib():
    """Load libglance.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; build it with "
                           "tree_verified_block_gb300._build.build() (nvcc, sm_103a)")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    st = ctypes.c_int
    L.glance_build_tree_workspace_bytes.argtypes = [i32, i32, i32]
    L.glance_build_tree_workspace_bytes.restype = sz
    L.glance_build_tree.argtypes = [vp, i32, i32, i32, i32, vp, vp, ctypes.POINTER(TreeC), vp, sz, vp]
    L.glance_build_tree.restype = st
    L.glance_tree_attention_workspace_bytes.argtypes = [i32, i32, ctypes.POINTER(KVC)]
    L.glance_tree_attention_workspace_bytes.restype = sz
    L.glance_tree_attention.argtypes = [vp, i32, ctypes.POINTER(KVC), ctypes.POINTER(TreeC),
                                        ctypes.c_float, vp, vp, sz, vp]
    L.glance_tree_attention.restype = st
    L.glance_tree_attention_timeout_check.argtypes = [vp, i32, ctypes.POINTER(KVC), ctypes.POINTER(TreeC),
                                                      ctypes.c_float, vp, vp, sz, ctypes.c_ulonglong, vp]
    L.glance_tree_attention_timeout_check.restype = st
    L.glance_lmhead_argmax_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.glance_lmhead_argmax_workspace_bytes.restype = sz
    L.glance_lmhead_argmax.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.glance_lmhead_argmax.restype = st
    L.glance_lmhead_argmax_noalloc.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp]
    L.glance_lmhead_argmax_noalloc.restype = st
    L.glance_lmhead_packed_w_bytes.argtypes = [i32, i32]
    L.glance_lmhead_packed_w_bytes.restype = sz
    L.glance_lmhead_pack_w.argtypes = [vp, i32, i32, vp, sz, vp]
    L.glance_lmhead_pack_w.restype = st
    L.glance_lmhead_argmax_packed.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp, sz, vp]
    L.glance_lmhead_argmax_packed.restype = st
    L.glance_accept_commit_workspace_bytes.argtypes = [i32]
    L.glance_accept_commit_workspace_bytes.restype = sz
    L.glance_accept_commit.argtypes = [ctypes.POINTER(TreeC), vp, ctypes.POINTER(KVC), i32, vp, vp,
                                       vp, vp, sz, vp]
    L.glance_accept_commit.restype = st
    L.glance_build_tree_batched_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.glance_build_tree_batched_workspace_bytes.restype = sz
    L.glance_build_tree_batched.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp,
                                            ctypes.POINTER(TreeC), vp, sz, vp]
    L.glance_build_tree_batched.restype = st
    L.glance_tree_attention_batched_workspace_bytes.argtypes = [i32, i32, i32, ctypes.POINTER(KVC)]
    L.glance_tree_attention_batched_workspace_bytes.restype = sz
    L.glance_tree_attention_batched.argtypes = [vp, i32, ctypes.POINTER(KVC), ctypes.POINTER(TreeC),
                                                i32, ctypes.c_float, vp, vp, sz, vp]
    L.glance_tree_attention_batched.restype = st
    L.glance_accept_commit_batched_workspace_bytes.argtypes = [i32, i32]
    L.glance_accept_commit_batched_workspace_bytes.restype = sz
    L.glance_accept_commit_batched.argtypes = [ctypes.POINTER(TreeC), i32, vp, ctypes.POINTER(KVC),
                                               i32, vp, vp, vp, vp, sz, vp]
    L.glance_accept_commit_batched.restype = st
    L.glance_lmhead_argmax_entropy.argtypes = [vp, vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]
    L.glance_lmhead_argmax_entropy.restype = st
    L.glance_build_tree_shared_workspace_bytes.argtypes = [i32, i32, i32, i32]
    L.glance_build_tree_shared_workspace_bytes.restype = sz
    L.glance_build_tree_shared.argtypes = [vp, i32, i32, i32, i32, i32, i32, vp, vp, vp,
                                           ctypes.c_float, ctypes.c_float, ctypes.POINTER(TreeC),
                                           vp, vp, sz, vp]
    L.glance_build_tree_shared.restype = st
    L.glance_row_sumsq.argtypes = [vp, i32, i32, vp, vp]
    L.glance_row_sumsq.restype = st
    L.glance_dense_qkv.argtypes = [vp, vp, i32, i32, i32, vp, i32, vp, vp, ctypes.c_float, vp,
                                   ctypes.c_float, vp, vp, vp]
    L.glance_dense_qkv.restype = st
    L.glance_dense_residual.argtypes = [vp, vp, i32, i32, i32, vp, vp, vp, vp]
    L.glance_dense_residual.restype = st
    L.glance_dense_swiglu.argtypes = [vp, vp, vp, i32, i32, i32, vp, i32, ctypes.c_float, vp, vp]
    L.glance_dense_swiglu.restype = st
    L.glance_lmhead_sample.argtypes = [vp, vp, i32, i32, i32, i32, ctypes.c_float, ctypes.c_uint64,
                                       vp, vp, vp, vp, vp, sz, vp]
    L.glance_lmhead_sample.restype = st
    L.glance_accept_commit_gated.argtypes = [ctypes.POINTER(TreeC), vp, vp, ctypes.c_float,
                                             ctypes.POINTER(KVC), i32, vp, vp, vp, vp, vp, sz, vp]
    L.glance_accept_commit_gated.restype = st
    L.glance_accept_commit_gated_batched.argtypes = [ctypes.POINTER(TreeC), i32, vp, vp,
                                                     ctypes.c_float, ctypes.POINTER(KVC), i32, vp,
                                                     vp, vp, vp, vp, sz, vp]
    L.glance_accept_commit_gated_batched.restype = st
    L.glance_rope_init.argtypes = [ctypes.POINTER(RopeC), i32, ctypes.c_double, i32, ctypes.POINTER(ctypes.c_int32), i32]
    L.glance_rope_init.restype = st
    L.glance_qk_norm_rope.argtypes = [vp, i32, i32, i32, ctypes.c_int64, i32, vp, vp, ctypes.c_float, vp, vp, vp, vp, vp]
    L.glance_qk_norm_rope.restype = st
    L.glance_kv4_write_rows.argtypes = [vp, vp, i32, i32, vp]
    L.glance_kv4_write_rows.restype = st
    L.glance_kv4_read_rows.argtypes = [vp, i32, i32, i32, vp, vp]
    L.glance_kv4_read_rows.restype = st
    L.glance_kv4_tree_attention_workspace_bytes.argtypes = [i32, i32, i32, vp]
    L.glance_kv4_tree_attention_workspace_bytes.restype = sz
    L.glance_kv4_tree_attention.argtypes = [vp, i32, vp, vp, i32, ctypes.c_float, vp, vp, sz, vp]
    L.glance_kv4_tree_attention.restype = st
    L.glance_kv4_accept_commit_workspace_bytes.argtypes = [i32, i32]
    L.glance_kv4_accept_commit_workspace_bytes.restype = sz
    L.glance_kv4_accept_commit.argtypes = [vp, i32, vp, vp, ctypes.c_float, vp, i32, vp, vp, vp, vp, vp, sz, vp]
    L.glance_kv4_accept_commit.restype = st
    i64, f32 = ctypes.c_int64, ctypes.c_float
    L.glance_q8_rows.argtypes = [vp, i64, i32, i32, i32, vp, i64, vp, vp]
    L.glance_q8_rows.restype = st
    L.glance_q8_norm_rows.argtypes = [vp, i64, vp, i64, i32, i32, i32, vp, f32, vp, i64, vp, i64, vp, vp]
    L.glance_q8_norm_rows.restype = st
    L.glance_q8_read_rows.argtypes = [vp, i64, vp, i32, i32, i32, vp, i64, vp]
    L.glance_q8_read_rows.restype = st
    L.glance_q8_linear.argtypes = [vp, i64, vp, i32, vp, i64, vp, i32, i32, i32, i32, vp, vp, i64, vp, i64, i32, vp]
    L.glance_q8_linear.restype = st
    L.glance_sample.argtypes = [vp, i64, i32, i32, i32, vp, vp, vp, vp, ctypes.c_uint64, vp, vp, vp, vp, vp]
    L.glance_sample.restype = st
    L.glance_last_error.argtypes = []
    L.glance_last_error.restype = ctypes.c_char_p
    L.glance_status_string.argtypes = [st]
    L.glance_status_string.restype = ctypes.c_char_p
    L.glance_device_status.argtypes = [ctypes.POINTER(ctypes.c_int32)]
    L.glance_device_status.restype = st
    L.glance_reset_device_status.argtypes = []
    L.glance_reset_device_status.restype = st
    L.glance_kv_write_rows.argtypes = [vp, ctypes.POINTER(KVC), i32, i32, vp]
    L.glance_kv_write_rows.restype = st
    L.glance_get_status.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
    L.glance_get_status.restype = st
    L.glance_clear_status.argtypes = [ctypes.c_void_p]
    L.glance_clear_status.restype = st
    L.glance_version.argtypes = []
    L.glance_version.restype = ctypes.c_int
    _lib = L
    return L


def _check(status):
    if status != 0:
        raise GlanceError(status, lib().glance_last_error().decode())


def _ptr(t):
    """Device pointer of a CUDA tensor (None for None). A host tensor would
    reach a kernel as an address it cannot read, so it is refused here."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("glance: every array argument must be a CUDA tensor (got one on %s)" % t.device)
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream, device):
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.bfloat16:
        return BF16
    raise TypeError(f"unsupported dtype {t.dtype}: float32 or bfloat16")


def workspace(nbytes, device="cuda"):
    """A zero-filled device workspace (the library leaves its counters at zero)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


class Tree:
    """Device arrays of one packed tree (N + 1 rows) and the C view of them."""

    def __init__(self, N, L, device="cuda"):
        rows = N + 1
        self.N, self.L, self.rows = N, L, rows
        self.mask_words = (rows + 63) // 64
        i32 = dict(dtype=torch.int32, device=device)
        self.token = torch.zeros(rows, **i32)
        self.parent = torch.zeros(rows, **i32)
        self.depth = torch.zeros(rows, **i32)
        self.pos_id = torch.zeros(rows, **i32)
        self.score = torch.zeros(rows, dtype=torch.float32, device=device)
        self.anc = torch.zeros((rows, self.mask_words), dtype=torch.int64, device=device)
        self.c = TreeC(N, L, self.mask_words, *(_ptr(t).value for t in (self.token, self.parent, self.depth,
                                                                            self.pos_id, self.score, self.anc)))

    def to_host(self):
        return dict(token=self.token.cpu().numpy(), parent=self.parent.cpu().numpy(),
                    depth=self.depth.cpu().numpy(), pos_id=self.pos_id.cpu().numpy(),
                    score=self.score.cpu().numpy(),
                    anc=self.anc.cpu().numpy().view("uint64"))


class KVLayer:
    """One layer's cache view: k, v tensors [n_kv_heads][t_cap][head_dim]."""

    def __init__(self, k, v, t_len):
        assert k.shape == v.shape and k.dim() == 3 and k.stride() == v.stride()
        assert k.stride(2) == 1, "head_dim must be contiguous"
        self.k, self.v, self.t_len = k, v, t_len
        Hkv, t_cap, D = k.shape
        self.c = KVC(_ptr(k).value, _ptr(v).value, _dtype_code(k), Hkv, D, t_cap,
                     k.stride(0), k.stride(1), _ptr(t_len).value)


class KV4Layer:
    """One layer's 4-bit cache view (include/glance.h, glance_kv4): codes k, v
    uint8 [n_kv_heads][t_cap][64] and their scales uint8 (or float8_e4m3fn)
    [n_kv_heads][t_cap][8], one factor for all of K and one for all of V."""

    def __init__(self, k, k_scale, v, v_scale, t_len, k_global=1.0, v_global=1.0):
        Hkv, t_cap, _ = k.shape
        heads = {t.stride(0) // w for t, w in ((k, 64), (k_scale, 8), (v, 64), (v_scale, 8))} if Hkv > 1 else {t_cap + t_cap % 2}
        for t, w in ((k, 64), (k_scale, 8), (v, 64), (v_scale, 8)):
            if t.shape != (Hkv, t_cap, w) or t.element_size() != 1 or t.stride(2) != 1 or t.stride(1) != w or (
                    Hkv > 1 and t.stride(0) % w):
                raise ValueError("glance: a 4-bit cache has one-byte codes [n_kv_heads, t_cap, 64] and scales "
                                 "[n_kv_heads, t_cap, 8] with whole rows next to each other")
            if t.device != k.device or t_len.device != k.device:
                raise ValueError("glance: codes, scales and t_len must be on one device")
        if len(heads) != 1:
            raise ValueError("glance: codes and scales need the same number of slots between heads")
        if Hkv == 1 and t_cap % 2:
            raise ValueError("glance: a 4-bit cache needs an even number of slots")
        if t_len.dtype != torch.int32 or t_len.numel() != 1:
            raise ValueError("glance: t_len must be one int32")
        self.k, self.k_scale, self.v, self.v_scale, self.t_len = k, k_scale, v, v_scale, t_len
        self.device = k.device
        self.c = KV4C(_ptr(k).value, _ptr(k_scale).value, _ptr(v).value, _ptr(v_scale).value, float(k_global),
                      float(v_global), Hkv, 128, t_cap, heads.pop(), _ptr(t_len).value)

    @classmethod
    def empty(cls, n_kv_heads, t_cap, t_len, k_global=1.0, v_global=1.0, device="cuda"):
        """A zero-filled cache of t_cap slots (rounded up to an even number)."""
        u8 = dict(dtype=torch.uint8, device=device)
        n = t_cap + t_cap % 2
        return cls(torch.zeros((n_kv_heads, n, 64), **u8), torch.zeros((n_kv_heads, n, 8), **u8),
                   torch.zeros((n_kv_heads, n, 64), **u8), torch.zeros((n_kv_heads, n, 8), **u8), t_len, k_global, v_global)


class Views(tuple):
    """Tree, KVLayer or KV4Layer objects of one device with their C array laid
    out once: calls that take a list of them accept it without building the
    array again. A tuple: the array points into the objects' tensors, so none
    may be added, exchanged or dropped."""

    def __init__(self, items):
        if not self:
            raise ValueError("glance: an empty list of views")
        if not all(isinstance(x, type(self[0])) and isinstance(x, (Tree, KVLayer, KV4Layer)) for x in self):
            raise TypeError("glance: views are Tree, KVLayer or KV4Layer objects, of one kind")
        on = {t.get_device() for x in self for t in ((x.anc,) if isinstance(x, Tree) else (x.k, x.v, x.t_len))}
        if len(on) != 1:
            raise ValueError("glance: every view of a list must be on one device")
        self.dev = on.pop()
        first = self[0].c
        self.c = (type(first) * len(self))(*[x.c for x in self])
        self.n, self.kind, self.at = len(self), type(self[0]), ctypes.addressof(self.c)
        self.heads = (self[0].rows, self[0].L) if isinstance(first, TreeC) else (first.n_kv_heads, first.head_dim)


class _Alone:
    """What a call needs to know of one view by itself: its C struct is an array
    of one. Kept with the view, so it must not refer to it: the caches of a view
    that is dropped are freed at once."""
    __slots__ = ("c", "at", "n", "kind", "dev", "heads")

    def __init__(self, view):
        checked = Views([view])
        self.c, self.at, self.n = view.c, ctypes.addressof(view.c), 1
        self.kind, self.dev, self.heads = checked.kind, checked.dev, checked.heads


def _views(x, kind):
    """x (a Views, a list of views, or one view) with its items checked, as a
    Views or, one view by itself, an _Alone."""
    if type(x) is Views and x.kind is kind:
        return x
    if isinstance(x, kind):
        alone = x.__dict__.get("_alone")
        if alone is None or alone.c is not x.c:
            alone = x._alone = _Alone(x)
        return alone
    if not isinstance(x, Views):
        x = Views(x if isinstance(x, (list, tuple)) else [x])
    if not issubclass(x.kind, kind):
        raise TypeError(f"glance: expected {kind.__name__} views, got {x.kind.__name__}")
    return x


def _i32(x, name):
    """x as an int32: ctypes would drop the bits above."""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"glance: {name} does not fit 32 bits")
    return x


class Rope:
    """Rotary positions as a plan (glance_rope_init): sections = how many of the
    head_dim / 2 frequencies each position axis turns (None: one axis)."""

    def __init__(self, head_dim, theta, sections=None, interleaved=False):
        self.c = RopeC()
        sec = [_i32(n, "a section") for n in (sections if sections is not None else [head_dim // 2])]
        _check(lib().glance_rope_init(ctypes.byref(self.c), _i32(head_dim, "head_dim"), float(theta), len(sec),
                                      (ctypes.c_int32 * len(sec))(*sec), int(bool(interleaved))))
        self.head_dim, self.n_axes, self.at = head_dim, len(sec), ctypes.addressof(self.c)


# ------------------------------------------------------------------- calls

def build_tree_workspace_bytes(L, V, N):
    return lib().glance_build_tree_workspace_bytes(L, V, N)


def build_tree(draft_logits, N, root_token, t_len, tree, ws, stream=None):
    L, V = draft_logits.shape
    assert draft_logits.is_contiguous()
    _check(lib().glance_build_tree(_ptr(draft_logits), _dtype_code(draft_logits), L, V, N,
                                   _ptr(root_token), _ptr(t_len), ctypes.byref(tree.c),
                                   _ptr(ws), ws.numel(), _stream(stream, draft_logits.device)))


def tree_attention_workspace_bytes(rows, n_q_heads, kv):
    return lib().glance_tree_attention_workspace_bytes(rows, n_q_heads, ctypes.byref(kv.c))


def tree_attention(q, kv, tree, scale, out, ws, stream=None):
    assert q.is_contiguous() and out.is_contiguous() and q.shape == out.shape
    _check(lib().glance_tree_attention(_ptr(q), q.shape[1], ctypes.byref(kv.c),
                                       ctypes.byref(tree.c), float(scale), _ptr(out), _ptr(ws),
                                       ws.numel(), _stream(stream, q.device)))


def tree_attention_timeout_check(q, kv, tree, scale, out, ws, wait_ns, stream=None):
    """The bf16 attention call with every pipeline wait limited to wait_ns and
    one key tile's V copy withheld: the kernel must set device status 4 and
    return (include/glance.h)."""
    assert q.is_contiguous() and out.is_contiguous() and q.shape == out.shape
    _check(lib().glance_tree_attention_timeout_check(_ptr(q), q.shape[1], ctypes.byref(kv.c),
                                                     ctypes.byref(tree.c), float(scale), _ptr(out),
                                                     _ptr(ws), ws.numel(), int(wait_ns),
                                                     _stream(stream, q.device)))


def lmhead_argmax_workspace_bytes(M, d, V, dtype):
    code = BF16 if dtype == torch.bfloat16 else F32
    return lib().glance_lmhead_argmax_workspace_bytes(M, d, V, code)


def lmhead_argmax(h, W, argmax, gap, maxlogit, ws, stream=None):
    M, d = h.shape
    assert W.shape[0] == d and h.is_contiguous() and W.is_contiguous() and h.dtype == W.dtype
    _check(lib().glance_lmhead_argmax(_ptr(h), _ptr(W), _dtype_code(h), M, d, W.shape[1],
                                      _ptr(argmax), _ptr(gap), _ptr(maxlogit), _ptr(ws),
                                      ws.numel(), _stream(stream, h.device)))


def lmhead_argmax_noalloc(h, W, argmax, gap, maxlogit, stream=None):
    """LM head + argmax for callers that cannot allocate: no workspace, the
    scratch lives in the library (calls on one device must not overlap)."""
    M, d = h.shape
    assert W.shape[0] == d and h.is_contiguous() and W.is_contiguous() and h.dtype == W.dtype
    _check(lib().glance_lmhead_argmax_noalloc(_ptr(h), _ptr(W), _dtype_code(h), M, d, W.shape[1],
                                              _ptr(argmax), _ptr(gap), _ptr(maxlogit),
                                              _stream(stream, h.device)))


def lmhead_packed_w_bytes(d, V):
    return lib().glance_lmhead_packed_w_bytes(d, V)


def lmhead_pack_w(W, W_packed, stream=None):
    """W (bf16 [d][V]) -> W_packed (any contiguous device tensor of at least
    lmhead_packed_w_bytes(d, V) bytes), the layout lmhead_argmax_packed reads."""
    d, V = W.shape
    assert W.is_contiguous() and W.dtype == torch.bfloat16 and W_packed.is_contiguous()
    _check(lib().glance_lmhead_pack_w(_ptr(W), d, V, _ptr(W_packed), W_packed.numel() * W_packed.element_size(),
                                      _stream(stream, W.device)))


def lmhead_argmax_packed(h, W_packed, V, argmax, gap, maxlogit, ws, stream=None):
    """lmhead_argmax (bf16, M <= 128) with W given as lmhead_pack_w wrote it."""
    M, d = h.shape
    assert h.is_contiguous() and h.dtype == torch.bfloat16 and W_packed.is_contiguous()
    _check(lib().glance_lmhead_argmax_packed(_ptr(h), _ptr(W_packed), M, d, V, _ptr(argmax), _ptr(gap),
                                             _ptr(maxlogit), _ptr(ws), ws.numel(), _stream(stream, h.device)))


def lmhead_argmax_entropy(h, W, argmax, gap, maxlogit, entropy, ws, stream=None):
    """lmhead_argmax plus each row's next-token entropy (nats), bf16."""
    M, d = h.shape
    assert W.shape[0] == d and h.is_contiguous() and W.is_contiguous() and h.dtype == W.dtype
    _check(lib().glance_lmhead_argmax_entropy(_ptr(h), _ptr(W), _dtype_code(h), M, d, W.shape[1],
                                              _ptr(argmax), _ptr(gap), _ptr(maxlogit),
                                              _ptr(entropy), _ptr(ws), ws.numel(),
                                              _stream(stream, h.device)))


def lmhead_sample(h, W, inv_temperature, seed, position, seq, tokens, gap, ws, stream=None):
    """Sampling-mode LM head: tokens[i] is a Gumbel-max draw from
    softmax(l_i / T), the noise keyed by (seed, position[i], seq[i])."""
    M, d = h.shape
    assert W.shape[0] == d and h.is_contiguous() and W.is_contiguous() and h.dtype == W.dtype
    _check(lib().glance_lmhead_sample(_ptr(h), _ptr(W), _dtype_code(h), M, d, W.shape[1],
                                      float(inv_temperature), int(seed) & ((1 << 64) - 1),
                                      _ptr(position), _ptr(seq), _ptr(tokens), _ptr(gap), _ptr(ws),
                                      ws.numel(), _stream(stream, h.device)))


def accept_commit_workspace_bytes(n_layers):
    return lib().glance_accept_commit_workspace_bytes(n_layers)


def accept_commit(tree, argmax, layers, n_accepted, accepted_tok, new_root, ws, stream=None):
    arr = (KVC * len(layers))(*[l.c for l in layers])
    _check(lib().glance_accept_commit(ctypes.byref(tree.c), _ptr(argmax), arr, len(layers),
                                      _ptr(n_accepted), _ptr(accepted_tok), _ptr(new_root),
                                      _ptr(ws), ws.numel(), _stream(stream, argmax.device)))


def accept_commit_gated(tree, argmax, gap, threshold, layers, n_accepted, accepted_tok, new_root,
                        gated, ws, stream=None):
    """accept_commit with the tie-aware gate on the rows' top-2 margins."""
    arr = (KVC * len(layers))(*[l.c for l in layers])
    _check(lib().glance_accept_commit_gated(ctypes.byref(tree.c), _ptr(argmax), _ptr(gap),
                                            float(threshold), arr, len(layers), _ptr(n_accepted),
                                            _ptr(accepted_tok), _ptr(new_root), _ptr(gated),
                                            _ptr(ws), ws.numel(), _stream(stream, argmax.device)))


# ------------------------------------------------------------ batched calls

def _trees(trees):
    if isinstance(trees, Views):
        return trees.c
    return (TreeC * len(trees))(*[t.c for t in trees])


def _kvs(kvs):
    if isinstance(kvs, Views):
        return kvs.c
    return (KVC * len(kvs))(*[k.c for k in kvs])


def build_tree_batched_workspace_bytes(B, L, V, N):
    return lib().glance_build_tree_batched_workspace_bytes(B, L, V, N)


def build_tree_batched(draft_logits, N, root_token, t_len, trees, ws, stream=None):
    """draft_logits [B][L][V]; root_token, t_len int32 [B]; trees: B Tree objects."""
    B, L, V = draft_logits.shape
    assert draft_logits.is_contiguous() and len(trees) == B
    _check(lib().glance_build_tree_batched(_ptr(draft_logits), _dtype_code(draft_logits), B, L, V,
                                           N, _ptr(root_token), _ptr(t_len), _trees(trees),
                                           _ptr(ws), ws.numel(),
                                           _stream(stream, draft_logits.device)))


def build_tree_shared_workspace_bytes(B, L, V, N_max):
    return lib().glance_build_tree_shared_workspace_bytes(B, L, V, N_max)


def build_tree_shared(draft_logits, N_max, N_total, root_token, t_len, trees, n_active, ws,
                      root_entropy=None, law_b0=0.0, law_b1=0.0, stream=None):
    """B trees under a shared budget of N_total nodes (at most N_max each); with
    root_entropy [B], node masses are keyed by the entropy law."""
    B, L, V = draft_logits.shape
    assert draft_logits.is_contiguous() and len(trees) == B
    _check(lib().glance_build_tree_shared(_ptr(draft_logits), _dtype_code(draft_logits), B, L, V,
                                          N_max, N_total, _ptr(root_token), _ptr(t_len),
                                          _ptr(root_entropy), float(law_b0), float(law_b1),
                                          _trees(trees), _ptr(n_active), _ptr(ws), ws.numel(),
                                          _stream(stream, draft_logits.device)))


def tree_attention_batched_workspace_bytes(rows, n_q_heads, kvs):
    return lib().glance_tree_attention_batched_workspace_bytes(len(kvs), rows, n_q_heads, _kvs(kvs))


def tree_attention_batched(q, kvs, trees, scale, out, ws, stream=None):
    """q, out [B][N+1][Hq][128] bf16; kvs: B KVLayer views of this layer."""
    B = q.shape[0]
    assert q.is_contiguous() and out.is_contiguous() and q.shape == out.shape
    assert len(kvs) == B and len(trees) == B
    _check(lib().glance_tree_attention_batched(_ptr(q), q.shape[2], _kvs(kvs), _trees(trees), B,
                                               float(scale), _ptr(out), _ptr(ws), ws.numel(),
                                               _stream(stream, q.device)))


def accept_commit_batched_workspace_bytes(B, n_layers):
    return lib().glance_accept_commit_batched_workspace_bytes(B, n_layers)


def accept_commit_batched(trees, argmax, layers, n_accepted, accepted_tok, new_root, ws,
                          stream=None):
    """layers[r][l]: KVLayer of request r, layer l; argmax [B][N+1]; outputs [B], [B][L], [B]."""
    B = len(trees)
    n_layers = len(layers[0])
    flat = [layers[r][l] for r in range(B) for l in range(n_layers)]
    _check(lib().glance_accept_commit_batched(_trees(trees), B, _ptr(argmax), _kvs(flat), n_layers,
                                              _ptr(n_accepted), _ptr(accepted_tok),
                                              _ptr(new_root), _ptr(ws), ws.numel(),
                                              _stream(stream, argmax.device)))


def accept_commit_gated_batched(trees, argmax, gap, threshold, layers, n_accepted, accepted_tok,
                                new_root, gated, ws, stream=None):
    B = len(trees)
    n_layers = len(layers[0])
    flat = [layers[r][l] for r in range(B) for l in range(n_layers)]
    _check(lib().glance_accept_commit_gated_batched(_trees(trees), B, _ptr(argmax), _ptr(gap),
                                                    float(threshold), _kvs(flat), n_layers,
                                                    _ptr(n_accepted), _ptr(accepted_tok),
                                                    _ptr(new_root), _ptr(gated), _ptr(ws),
                                                    ws.numel(), _stream(stream, argmax.device)))


# -------------------------------------------------------------- dense layers

def row_sumsq(x, sumsq, stream=None):
    """sumsq [M] (float32) = row sums of squares of x [M][d] (bf16)."""
    M, d = x.shape
    assert x.is_contiguous()
    _check(lib().glance_row_sumsq(_ptr(x), M, d, _ptr(sumsq), _stream(stream, x.device)))


def _n_parts(in_sumsq, M):
    if in_sumsq is None:
        return 0
    assert in_sumsq.dtype == torch.float32 and in_sumsq.is_contiguous() and in_sumsq.numel() % M == 0
    return in_sumsq.numel() // M


def dense_qkv(h, W_qkv, n_q_heads, in_sumsq, q_norm, k_norm, eps, pos_id, rope_theta, q_out, kv,
              stream=None):
    """in_sumsq: [n][M] partial row sums of squares of h (None: no input norm)."""
    M, d = h.shape
    assert h.is_contiguous() and W_qkv.is_contiguous() and q_out.is_contiguous()
    _check(lib().glance_dense_qkv(_ptr(h), _ptr(W_qkv), M, d, n_q_heads, _ptr(in_sumsq),
                                  _n_parts(in_sumsq, M), _ptr(q_norm), _ptr(k_norm), float(eps),
                                  _ptr(pos_id), float(rope_theta), _ptr(q_out), ctypes.byref(kv.c),
                                  _stream(stream, h.device)))


def dense_residual(x, W, residual, out, out_sumsq=None, stream=None):
    """out_sumsq: [N / 256][M] float32 to receive the output rows' sums of squares, or None."""
    M, K = x.shape
    N = W.shape[1]
    assert x.is_contiguous() and W.is_contiguous() and residual.is_contiguous() and out.is_contiguous()
    if out_sumsq is not None:
        assert out_sumsq.dtype == torch.float32 and out_sumsq.numel() >= (N // 256) * M
    _check(lib().glance_dense_residual(_ptr(x), _ptr(W), M, K, N, _ptr(residual), _ptr(out),
                                       _ptr(out_sumsq), _stream(stream, x.device)))


def dense_swiglu(h, W_gate, W_up, in_sumsq, eps, act, stream=None):
    M, d = h.shape
    inter = W_gate.shape[1]
    assert h.is_contiguous() and W_gate.is_contiguous() and W_up.is_contiguous() and act.is_contiguous()
    _check(lib().glance_dense_swiglu(_ptr(h), _ptr(W_gate), _ptr(W_up), M, d, inter, _ptr(in_sumsq),
                                     _n_parts(in_sumsq, M), float(eps), _ptr(act),
                                     _stream(stream, h.device)))


# ------------------------------------------- norm + rotary, 4-bit caches

_DTYPES = {torch.float32: F32, torch.bfloat16: BF16}
_I32, _F32T, _BF16T = torch.int32, torch.float32, torch.bfloat16


def _on(stream, dev):
    """The stream to launch on: the given one, else the device's current one.
    The device must be the current one."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError("glance: the tensors are not on the current device")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _workspace(ws, dev):
    """Address of a call's workspace: bytes that lie next to each other (an
    expanded tensor counts bytes that it does not have)."""
    if not ws.is_contiguous():
        raise ValueError("glance: the workspace must be contiguous")
    if ws.get_device() != dev:
        raise _elsewhere()
    return ws.data_ptr()


def _elsewhere():
    return ValueError("glance: every array argument must be a CUDA tensor of one device")


def qk_norm_rope(qkv, n_q_heads, q_norm, k_norm, eps, pos, rope, q_out, kv, stream=None):
    """qkv [B * M][(Hq + 2 Hkv) * D] (rows may be strided) -> per-head RMS norm
    of q and k, rotary position, q to q_out [B * M][Hq][D], k and v to slots
    T.. of kv (one KVLayer, or B of them). pos int32 [n_axes][B * M]."""
    kv = _views(kv, KVLayer)
    B, dev, (Hkv, D), shape, dtype = kv.n, kv.dev, kv.heads, qkv.shape, qkv.dtype
    rows, (step, unit) = shape[0], qkv.stride() if len(shape) == 2 else (0, 0)
    if unit != 1 or rows % B or shape[1] != (n_q_heads + 2 * Hkv) * D or rope.head_dim != D:
        raise ValueError("glance: qkv must be [B * M, (n_q_heads + 2 * n_kv_heads) * head_dim], rope and kv of its head_dim")
    if dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {dtype}: float32 or bfloat16")
    if pos.dtype is not _I32 or pos.shape[-1] != rows or pos.numel() != rope.n_axes * rows or not pos.is_contiguous():
        raise ValueError("glance: pos must be contiguous int32 [n_axes, B * M]")
    if q_out.dtype is not dtype or q_out.numel() != rows * n_q_heads * D or not q_out.is_contiguous():
        raise ValueError("glance: q_out must be contiguous [B * M, n_q_heads, head_dim] of qkv's dtype")
    if qkv.get_device() != dev or pos.get_device() != dev or q_out.get_device() != dev:
        raise _elsewhere()
    _check(lib().glance_qk_norm_rope(qkv.data_ptr(), _DTYPES[dtype], B, rows // B, step if rows > 1 else shape[1], n_q_heads,
                                     None if q_norm is None else _norm(q_norm, D, dev),
                                     None if k_norm is None else _norm(k_norm, D, dev), eps, pos.data_ptr(), rope.at,
                                     q_out.data_ptr(), kv.at, _on(stream, dev)))


def _norm(w, D, dev):
    if w.dtype is not _F32T or w.numel() != D or not w.is_contiguous():
        raise ValueError("glance: norm weights must be contiguous float32 [head_dim]")
    if w.get_device() != dev:
        raise _elsewhere()
    return w.data_ptr()


def _rows16(x, layers, rows):
    if x.dtype is not _BF16T or not x.is_contiguous() or x.shape != (layers.n, 2, layers.heads[0], rows, 128):
        raise ValueError("glance: rows must be contiguous bfloat16 [n_layers, 2, n_kv_heads, rows, 128]")
    if x.get_device() != layers.dev:
        raise _elsewhere()
    return x.data_ptr()


def kv4_write_rows(src, layers, rows, stream=None):
    """Quantise src [n_layers, 2, n_kv_heads, rows, 128] (bf16, K before V) into
    every layer's 4-bit cache at slots T..T+rows-1 (T read on the device)."""
    layers = _views(layers, KV4Layer)
    _check(lib().glance_kv4_write_rows(_rows16(src, layers, rows), layers.at, layers.n, rows, _on(stream, layers.dev)))


def kv4_read_rows(layers, first, rows, dst, stream=None):
    """dst [n_layers, 2, n_kv_heads, rows, 128] (bf16) = the values of slots
    first .. first + rows - 1 of every layer's 4-bit cache."""
    layers = _views(layers, KV4Layer)
    _check(lib().glance_kv4_read_rows(layers.at, layers.n, _i32(first, "first"), rows, _rows16(dst, layers, rows), _on(stream, layers.dev)))


def kv4_tree_attention_workspace_bytes(rows, n_q_heads, kvs):
    kvs = _views(kvs, KV4Layer)
    return lib().glance_kv4_tree_attention_workspace_bytes(kvs.n, _i32(rows, "rows"), _i32(n_q_heads, "n_q_heads"), kvs.at)


_DECODE = {}


def kv4_tree_attention(q, kvs, trees, scale, out, ws, stream=None):
    """Tree attention over 4-bit caches: q, out [B][N+1][Hq][128] bf16 (B = 1:
    [N+1][Hq][128] too), kvs B KV4Layer views, trees B Tree objects. trees
    None: plain decoding, one row per request that sees the prefix and itself."""
    kvs = _views(kvs, KV4Layer)
    B, dev, shape = kvs.n, kvs.dev, q.shape
    rows, heads = shape[-3], shape[-2]
    if q.dtype is not _BF16T or out.dtype is not _BF16T or not q.is_contiguous() or not out.is_contiguous() \
            or shape != out.shape or shape[-1] != 128 or q.numel() != B * rows * heads * 128:
        raise ValueError("glance: q and out must be contiguous bfloat16 [B, N + 1, n_q_heads, 128]")
    if trees is None:
        c = _DECODE.get(B)
        if c is None:
            c = _DECODE[B] = (TreeC * B)(*[TreeC(0, 1, 1) for _ in range(B)])
        c = ctypes.addressof(c)
        if rows != 1:
            raise ValueError("glance: without trees q has one row per request")
    else:
        trees = _views(trees, Tree)
        if trees.n != B or trees.heads[0] != rows:
            raise ValueError("glance: need one tree of q's N + 1 rows per request")
        if trees.dev != dev:
            raise _elsewhere()
        c = trees.at
    if q.get_device() != dev or out.get_device() != dev:
        raise _elsewhere()
    _check(lib().glance_kv4_tree_attention(q.data_ptr(), heads, kvs.at, c, B, scale, out.data_ptr(), _workspace(ws, dev), ws.nbytes,
                                           _on(stream, dev)))


def kv4_accept_commit_workspace_bytes(B, n_layers):
    return lib().glance_kv4_accept_commit_workspace_bytes(_i32(B, "B"), _i32(n_layers, "n_layers"))


def _array(x, dtype, n, dev):
    if x.dtype is not dtype or x.numel() < n or not x.is_contiguous():
        raise ValueError("glance: argmax, n_accepted, accepted_tok, new_root and gated must be contiguous int32 [B, N + 1], [B], "
                         "[B, L], [B], [B], gap contiguous float32 [B, N + 1]")
    if x.get_device() != dev:
        raise _elsewhere()
    return x.data_ptr()


def kv4_accept_commit(trees, argmax, layers, n_accepted, accepted_tok, new_root, ws, gap=None, gate_threshold=0.0,
                      gated=None, stream=None):
    """Walk + commit on 4-bit caches: trees B Tree objects (or one), layers the
    B * n_layers KV4Layer views (request-major), argmax [B][N+1], outputs [B],
    [B][L], [B]. With gap [B][N+1] and gated [B]: the tie-aware gate."""
    trees, layers = _views(trees, Tree), _views(layers, KV4Layer)
    B, dev, (rows, L) = trees.n, layers.dev, trees.heads
    if layers.n % B:
        raise ValueError("glance: layers must hold the same number of views for every request")
    if trees.dev != dev:
        raise _elsewhere()
    _check(lib().glance_kv4_accept_commit(trees.at, B, _array(argmax, _I32, B * rows, dev),
                                          None if gap is None else _array(gap, _F32T, B * rows, dev), gate_threshold, layers.at,
                                          layers.n // B, _array(n_accepted, _I32, B, dev), _array(accepted_tok, _I32, B * L, dev),
                                          _array(new_root, _I32, B, dev),
                                          None if gated is None else _array(gated, _I32, B, dev), _workspace(ws, dev), ws.nbytes,
                                          _on(stream, dev)))


# ------------------------------------------------------------- 8-bit rows

_CODES = (torch.uint8, torch.float8_e4m3fn)
ACTS = {"none": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def _bad(what):
    return ValueError("glance: " + what)


def _matrix(x, shape, what, dev):
    """(address, elements between rows) of a matrix whose rows lie in one piece each."""
    if x.shape != shape:
        raise _bad(what)
    step, unit = x.stride()
    if unit != 1:
        raise _bad(what)
    if x.get_device() != dev:
        raise _elsewhere()
    return x.data_ptr(), step if shape[0] > 1 else shape[1]


def _floats(x, n, what, dev):
    if x.dtype is not _F32T or x.numel() != n or not x.is_contiguous():
        raise _bad(what)
    if x.get_device() != dev:
        raise _elsewhere()
    return x.data_ptr()


def _codes(x, shape, what, dev):
    if x.dtype not in _CODES:
        raise _bad(what)
    return _matrix(x, shape, what, dev)


_CODES_TEXT = "codes must be uint8 or float8_e4m3fn of the rows' shape"
_SCALES_TEXT = "scales must be contiguous float32, one per row"
_ROWS_TEXT = "x, residual and total must be float32 or bfloat16 [M, d], all of one type"


def _rows_of(x, what):
    """(shape, type's number) of a matrix of floats."""
    shape, dtype = x.shape, _DTYPES.get(x.dtype)
    if dtype is None or len(shape) != 2:
        raise _bad(what)
    return shape, dtype


def q8_rows(x, codes, scales, stream=None):
    """codes (uint8 or float8_e4m3fn [M, d]), scales (float32 [M]) <- rows of x [M, d]: e4m3 with a power-of-two scale per row."""
    dev, (shape, dtype) = x.get_device(), _rows_of(x, _ROWS_TEXT)
    (xp, xs), (cp, cs) = _matrix(x, shape, _ROWS_TEXT, dev), _codes(codes, shape, _CODES_TEXT, dev)
    _check(lib().glance_q8_rows(xp, xs, dtype, shape[0], shape[1], cp, cs, _floats(scales, shape[0], _SCALES_TEXT, dev), _on(stream, dev)))


def q8_norm_rows(x, residual, weight, eps, total, codes, scales, stream=None):
    """total <- x + residual (either None; total may be x or residual), codes and scales <- its RMS-normed rows times weight
    (float32 [d] or None), in e4m3 with a power-of-two scale per row."""
    dev, (shape, dtype) = x.get_device(), _rows_of(x, _ROWS_TEXT)
    (M, d), one = shape, x.dtype
    (xp, xs), (cp, cs) = _matrix(x, shape, _ROWS_TEXT, dev), _codes(codes, shape, _CODES_TEXT, dev)
    rp, rs, tp, ts = None, 0, None, 0
    if residual is not None:
        if residual.dtype is not one:
            raise _bad(_ROWS_TEXT)
        rp, rs = _matrix(residual, shape, _ROWS_TEXT, dev)
    if total is not None:
        if total.dtype is not one:
            raise _bad(_ROWS_TEXT)
        tp, ts = _matrix(total, shape, _ROWS_TEXT, dev)
    _check(lib().glance_q8_norm_rows(xp, xs, rp, rs, dtype, M, d,
                                     None if weight is None else _floats(weight, d, "weight must be contiguous float32 [d]", dev),
                                     eps, tp, ts, cp, cs, _floats(scales, M, _SCALES_TEXT, dev), _on(stream, dev)))


def q8_read_rows(codes, scales, out, stream=None):
    """out [M, d] (float32 or bfloat16) = code * scale."""
    dev, (shape, dtype) = out.get_device(), _rows_of(out, _ROWS_TEXT)
    (op, os_), (cp, cs) = _matrix(out, shape, _ROWS_TEXT, dev), _codes(codes, shape, _CODES_TEXT, dev)
    _check(lib().glance_q8_read_rows(cp, cs, _floats(scales, shape[0], _SCALES_TEXT, dev), dtype, shape[0], shape[1], op, os_,
                                     _on(stream, dev)))


def q8_linear(x, x_scale, w, w_scale, out, bias=None, act="none", gated=False, residual=None, stream=None):
    """out [M, N] (float32 or bfloat16) = act(x_scale x . w w_scale + bias) + residual: x [M, K] and w [N, K] codes of the row
    calls (or any e4m3), w_scale and bias float32 [N]. gated: w [2 N, K], gate rows then up rows, out = act(gate) * up."""
    dev, (shape, dtype) = out.get_device(), _rows_of(out, "out must be float32 or bfloat16 [M, N]")
    (M, N), K = shape, x.shape[-1]
    rows, kind = 2 * N if gated else N, ACTS.get(act)
    if kind is None:
        raise _bad("act must be one of " + ", ".join(ACTS))
    (op, os_), (xp, xs) = _matrix(out, shape, "out must have its rows in one piece each", dev), _codes(
        x, (M, K), "x must be uint8 or float8_e4m3fn [M, K]", dev)
    wp, wst = _codes(w, (rows, K), "w must be uint8 or float8_e4m3fn [N, K] (gated: [2 N, K])", dev)
    rp, rs = None, 0
    if residual is not None:
        if residual.dtype is not out.dtype:
            raise _bad("residual must be of out's shape and type")
        rp, rs = _matrix(residual, shape, "residual must be of out's shape and type", dev)
    _check(lib().glance_q8_linear(xp, xs, _floats(x_scale, M, "x_scale must be contiguous float32 [M]", dev), M, wp, wst,
                                  _floats(w_scale, rows, "w_scale must be contiguous float32, one per row of w", dev), N, K, 1 if gated else 0,
                                  kind, None if bias is None else _floats(bias, rows, "bias must be contiguous float32, one per row of w", dev),
                                  rp, rs, op, os_, dtype, _on(stream, dev)))


def _per_row(x, dtype, M, dev):
    if x is None:
        return None
    if x.dtype is not dtype or x.numel() != M or not x.is_contiguous():
        raise ValueError("glance: temperature, top_p, min_p and gap must be contiguous float32, top_k, position, seq and tokens "
                         "contiguous int32, one per row of logits")
    if x.get_device() != dev:
        raise _elsewhere()
    return x.data_ptr()


def sample(logits, temperature, top_k, top_p, min_p, seed, position, seq, tokens, gap=None, stream=None):
    """tokens (int32 [M]) drawn from rows of logits [M, V] (float32 or bfloat16) with each row's temperature (0: argmax), top_k,
    top_p and min_p (tensors [M] or None), the noise keyed by (seed, position[row], seq[row]) as in lmhead_sample."""
    dev, (shape, dtype) = logits.get_device(), _rows_of(logits, "logits must be float32 or bfloat16 [M, V]")
    (M, V), (lp, ls) = shape, _matrix(logits, shape, "logits must have their rows in one piece each", dev)
    if position is None or tokens is None:
        raise ValueError("glance: position and tokens are required")
    _check(lib().glance_sample(lp, ls, dtype, M, V, _per_row(temperature, _F32T, M, dev), _per_row(top_k, _I32, M, dev),
                               _per_row(top_p, _F32T, M, dev), _per_row(min_p, _F32T, M, dev), int(seed) & ((1 << 64) - 1),
                               _per_row(position, _I32, M, dev), _per_row(seq, _I32, M, dev), _per_row(tokens, _I32, M, dev),
                               _per_row(gap, _F32T, M, dev), _on(stream, dev)))


def device_status():
    """(code, text) of the device status word; synchronises the device."""
    code = ctypes.c_int32(0)
    lib().glance_device_status(ctypes.byref(code))
    return code.value, DEV_STATUS.get(code.value, "unknown")


def reset_device_status():
    _check(lib().glance_reset_device_status())


def kv_write_rows(src, layers, rows, stream=None):
    """Scatter src [n_layers, 2, n_kv_heads, rows, head_dim] (K before V) into
    every layer's cache at slots T..T+rows-1 (T read on the device)."""
    assert src.is_contiguous()
    arr = (KVC * len(layers))(*[l.c for l in layers])
    _check(lib().glance_kv_write_rows(_ptr(src), arr, len(layers), int(rows), _stream(stream, src.device)))


STATUS_WORDS = 6


def get_status(out, stream=None):
    """Enqueue the stream-ordered status read: out (int32 [6], CUDA or pinned
    host tensor) gets the first non-zero word in out[0] and the words of the
    tree build, attention, LM head, commit and dense kernels in out[1..5]."""
    assert out.dtype == torch.int32 and out.numel() >= STATUS_WORDS and out.is_contiguous()
    if not (out.is_cuda or out.is_pinned()):
        raise ValueError("glance: get_status needs a CUDA or pinned host tensor")
    dev = out.device if out.is_cuda else torch.device("cuda", torch.cuda.current_device())
    _check(lib().glance_get_status(ctypes.c_void_p(out.data_ptr()), _stream(stream, dev)))


def clear_status(stream=None, device=None):
    """Enqueue a clear of every device status word on the stream."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    _check(lib().glance_clear_status(_stream(stream, dev)))


def version():
    return lib().glance_version()
