"""ctypes binding of the 4-bit paged key/value cache C-ABI (include/kvcache.h).

Argument marshalling only: every step runs in libagemm.so's kernels, and the
binding raises when the library is missing.
"""
from __future__ import annotations

import ctypes
import struct

from . import agemm
from .agemm import OK, AgemmError, status_string

EXPORTED = (
    "kvc_create", "kvc_destroy", "kvc_page_bytes", "kvc_append", "kvc_attend", "kvc_attend_workspace", "kvc_read",
    "kvc_check", "kvc_last_error", "kvc_tree", "kvc_attend_tree", "kvc_verify", "kvc_verify_workspace", "kvc_commit",
)

_vp, _i32, _i64, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float


class AppendArgs(ctypes.Structure):
    """kvc_append_args."""
    _fields_ = [("tokens", _i64), ("q", _vp), ("k", _vp), ("v", _vp), ("q_out", _vp),
                ("q_token_stride", _i64), ("q_head_stride", _i64), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_token_stride", _i64), ("v_head_stride", _i64), ("out_token_stride", _i64),
                ("out_head_stride", _i64), ("slots", _vp), ("positions", _vp), ("rope", _vp), ("rope_len", _i64),
                ("rope_dims", _i32), ("interleaved", _i32), ("q_norm", _vp), ("k_norm", _vp), ("eps", _f32)]


class AttendArgs(ctypes.Structure):
    """kvc_attend_args."""
    _fields_ = [("batch", _i32), ("max_q", _i32), ("tokens", _i64), ("q", _vp), ("q_token_stride", _i64),
                ("q_head_stride", _i64), ("q_start", _vp), ("kv_len", _vp), ("q_off", _vp), ("page_table", _vp),
                ("table_stride", _i64), ("table_width", _i32), ("causal", _i32), ("max_kv", _i64), ("scale", _f32),
                ("out_f32", _i32), ("out", _vp), ("lse", _vp)]


class TreeArgs(ctypes.Structure):
    """kvc_tree_args."""
    _fields_ = [("batch", _i32), ("max_q", _i32), ("tokens", _i64), ("q_start", _vp), ("kv_len", _vp), ("parent", _vp),
                ("page_table", _vp), ("table_stride", _i64), ("table_width", _i32), ("mask_words", _i32), ("mask", _vp),
                ("positions", _vp), ("slots", _vp), ("total_len", _vp)]


class VerifyArgs(ctypes.Structure):
    """kvc_verify_args."""
    _fields_ = [("batch", _i32), ("max_q", _i32), ("tokens", _i64), ("q_start", _vp), ("parent", _vp), ("token", _vp),
                ("p", _vp), ("q", _vp), ("p_stride", _i64), ("q_stride", _i64), ("vocab", _i64), ("u", _vp),
                ("max_children", _i32), ("path", _vp), ("count", _vp), ("next", _vp)]


class CommitArgs(ctypes.Structure):
    """kvc_commit_args."""
    _fields_ = [("batch", _i32), ("max_q", _i32), ("tokens", _i64), ("q_start", _vp), ("kv_len", _vp), ("path", _vp),
                ("count", _vp), ("page_table", _vp), ("table_stride", _i64), ("table_width", _i32), ("new_len", _vp)]


# The same structs as bytes: packing them costs a third of filling a ctypes.Structure, and these calls are made for
# every layer of a decode step. Null pointers are 0.
_CODE = {_vp: "P", _i32: "i", _i64: "q", _f32: "f"}
_pack_append, _pack_attend, _pack_tree, _pack_verify, _pack_commit = (
    struct.Struct("@" + "".join(_CODE[t] for _, t in st._fields_)).pack
    for st in (AppendArgs, AttendArgs, TreeArgs, VerifyArgs, CommitArgs))

_ready = False


def load() -> ctypes.CDLL:
    """libagemm.so with the kvc_* signatures set."""
    global _ready
    lib = agemm.load()
    if not _ready:
        lib.kvc_create.argtypes = [ctypes.POINTER(_vp), ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, _i64]
        lib.kvc_destroy.argtypes = [_vp]
        lib.kvc_page_bytes.argtypes = [_vp, ctypes.POINTER(_i64)]
        lib.kvc_append.argtypes = [_vp, _vp, _vp, _vp]  # a packed AppendArgs
        lib.kvc_attend.argtypes = [_vp, _vp, _vp, _vp, _i64, _vp]  # a packed AttendArgs
        lib.kvc_attend_workspace.argtypes = [_vp, _i32, _i32, _i64, ctypes.POINTER(_i64)]
        lib.kvc_attend_tree.argtypes = [_vp, _vp, _vp, _vp, _i32, _vp, _i64, _vp]  # a packed AttendArgs
        lib.kvc_tree.argtypes = [_vp, _vp, _vp]  # a packed TreeArgs
        lib.kvc_verify.argtypes = [_vp, _vp, _vp, _i64, _vp]  # a packed VerifyArgs
        lib.kvc_verify_workspace.argtypes = [_vp, _i32, _i64, ctypes.POINTER(_i64)]
        lib.kvc_commit.argtypes = [_vp, _vp, _i32, _vp, _vp]  # page pointers, a packed CommitArgs
        lib.kvc_read.argtypes = [_vp, _vp, _i64, _vp, _vp, _vp, _vp]
        lib.kvc_check.argtypes = [_vp]
        lib.kvc_last_error.argtypes = [_vp]
        lib.kvc_last_error.restype = ctypes.c_char_p
        for name in EXPORTED:
            if name != "kvc_last_error":
                getattr(lib, name).restype = ctypes.c_int
        _ready = True
    return lib


class KvCache:
    """One shape of the 4-bit paged cache: Hq query heads on Hkv key/value heads of D channels.

    The context owns no device memory: pages (``new_pages``) and the attention's
    workspace (``workspace``) are the caller's tensors. Matrices are float16
    with contiguous channels; outputs are given by the caller."""

    def __init__(self, Hq: int, Hkv: int, D: int, page_tokens: int = 64, num_pages: int = 1):
        import torch
        lib = load()
        self._lib = lib
        self.Hq, self.Hkv, self.D = int(Hq), int(Hkv), int(D)
        self.page_tokens, self.num_pages = int(page_tokens), int(num_pages)
        h = _vp()
        rc = lib.kvc_create(ctypes.byref(h), self.Hq, self.Hkv, self.D, self.page_tokens, self.num_pages)
        if rc != OK:
            raise AgemmError(rc, f"kvc_create: {status_string(rc)}")
        self._h = h
        self._index = torch.cuda.current_device()
        self.device = torch.device("cuda", self._index)
        n = _i64()
        lib.kvc_page_bytes(h, ctypes.byref(n))
        self.page_bytes = n.value
        self._f16, self._f32 = torch.float16, torch.float32
        self._i32, self._i64, self._u8 = torch.int32, torch.int64, torch.uint8
        self._pages_shape, self._D = (self.num_pages, self.page_bytes), (self.D,)
        self._current = torch._C._cuda_getCurrentRawStream

    # -- helpers
    def _raise(self, rc: int, what: str):
        if rc != OK:
            msg = self._lib.kvc_last_error(self._h).decode()
            raise AgemmError(rc, f"{what}: {msg or status_string(rc)}")

    def _stream(self, stream):
        return stream.cuda_stream if stream is not None else self._current(self._index)

    def _plain(self, t, what, dtype, shape):
        """Pointer of a contiguous tensor of this context's device."""
        if t.dtype is not dtype or t.get_device() != self._index:
            raise TypeError(f"{what} must be a {dtype} tensor on {self.device}")
        if t.shape != shape:
            raise ValueError(f"{what} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{what} must be contiguous")
        return t.data_ptr()

    def _heads(self, t, what, T, H):
        """Pointer, token and head stride of a (T, H, D) float16 tensor with contiguous channels."""
        if t.dtype is not self._f16 or t.get_device() != self._index:
            raise TypeError(f"{what} must be a float16 tensor on {self.device}")
        if t.shape != (T, H, self.D):
            raise ValueError(f"{what} must have shape {(T, H, self.D)}, got {tuple(t.shape)}")
        st, sh, sd = t.stride()
        if sd != 1:
            raise ValueError(f"{what} must have contiguous channels")
        return t.data_ptr(), st if T > 1 else H * self.D, sh if H > 1 else self.D

    def _table(self, page_table, B):
        """Pointer, row stride and width of a (B, width) int32 page table."""
        if page_table.dtype is not self._i32 or page_table.get_device() != self._index or page_table.dim() != 2:
            raise TypeError(f"page_table must be a two-dimensional int32 tensor on {self.device}")
        rows, W = page_table.shape
        if rows != B:
            raise ValueError(f"page_table must have {B} rows, got {rows}")
        ts, ws = page_table.stride()
        if W > 1 and ws != 1:
            raise ValueError("page_table must have contiguous rows")
        return page_table.data_ptr(), ts if B > 1 else W, W

    def _probabilities(self, t, what, T):
        """Pointer, row stride and vocabulary of a (T, V) float32 tensor with contiguous rows."""
        if t.dtype is not self._f32 or t.get_device() != self._index or t.dim() != 2:
            raise TypeError(f"{what} must be a two-dimensional float32 tensor on {self.device}")
        rows, V = t.shape
        if rows != T:
            raise ValueError(f"{what} must have {T} rows, got {rows}")
        st, sv = t.stride()
        if V > 1 and sv != 1:
            raise ValueError(f"{what} must have contiguous rows")
        return t.data_ptr(), st if T > 1 else V, V

    def _bytes(self, workspace):
        if workspace.dtype is not self._u8 or workspace.get_device() != self._index or not workspace.is_contiguous():
            raise TypeError(f"workspace must be a contiguous uint8 tensor on {self.device}")
        return workspace

    def _pages(self, pages):
        return self._plain(pages, "pages", self._u8, self._pages_shape)

    # -- memory of the caller
    def new_pages(self):
        """Zeroed pages: a (num_pages, page_bytes) uint8 tensor."""
        import torch
        return torch.zeros(self.num_pages, self.page_bytes, dtype=torch.uint8, device=self.device)

    def workspace(self, batch: int, max_q: int = 1, max_kv: int = 1):
        """Workspace for every ``attend`` call within these bounds (smaller batches, chunks and lengths too): one for
        each call that may run at the same time."""
        import torch
        n = _i64()
        rc = self._lib.kvc_attend_workspace(self._h, int(batch), int(max_q), int(max_kv), ctypes.byref(n))
        if rc != OK:
            raise AgemmError(rc, f"kvc_attend_workspace: {status_string(rc)}")
        return torch.empty(max(16, n.value), dtype=torch.uint8, device=self.device)

    # -- the C-ABI
    def append(self, pages, q=None, k=None, v=None, slots=None, positions=None, rope=None, interleaved: bool = False,
               q_norm=None, k_norm=None, eps: float = 1e-6, q_out=None, stream=None):
        """kvc_append: q_out = rope(norm(q)); rope(norm(k)) and v to their slots in 4 bits.

        q (T, Hq, D), k and v (T, Hkv, D), strided rows allowed; slots and positions (T,) int64;
        rope (rope_len, rope_dims) float32, cosines then sines; norm weights (D,) float16."""
        if q is None and k is None:
            raise ValueError("neither q nor k given")
        T = (q if q is not None else k).shape[0]
        plain = self._plain
        qp = op = kp = vp = rp = sp = pp = qw = kw = 0
        qt = qh = ot = oh = kt = kh = vt = vh = rl = rd = 0
        if q is not None:
            qp, qt, qh = self._heads(q, "q", T, self.Hq)
            if q_out is not None:
                op, ot, oh = self._heads(q_out, "q_out", T, self.Hq)
        if k is not None:
            kp, kt, kh = self._heads(k, "k", T, self.Hkv)
        if v is not None:
            vp, vt, vh = self._heads(v, "v", T, self.Hkv)
        if slots is not None:
            sp = plain(slots, "slots", self._i64, (T,))
        if rope is not None:
            rl, rd = rope.shape
            rp = plain(rope, "rope", self._f32, (rl, rd))
        if positions is not None:
            pp = plain(positions, "positions", self._i64, (T,))
        if q_norm is not None:
            qw = plain(q_norm, "q_norm", self._f16, self._D)
        if k_norm is not None:
            kw = plain(k_norm, "k_norm", self._f16, self._D)
        args = _pack_append(T, qp, kp, vp, op, qt, qh, kt, kh, vt, vh, ot, oh, sp, pp, rp, rl, rd, bool(interleaved),
                            qw, kw, eps)
        rc = self._lib.kvc_append(self._h, self._pages(pages) if pages is not None else None, args, self._stream(stream))
        if rc != OK:
            self._raise(rc, "kvc_append")

    def attend(self, pages, q, kv_len, page_table, out, lse=None, q_start=None, max_q: int = 1, q_off=None,
               causal: bool = True, scale: float | None = None, max_kv: int | None = None, workspace=None, stream=None,
               tree=None):
        """kvc_attend: attention of q (T, Hq, D) over the cached tokens of each sequence into out (T, Hq, D)
        float16 or float32 and lse (T, Hq) float32. With tree (T, words) int64, the masks that ``tree`` makes,
        kvc_attend_tree: each query sees the first q_off tokens and the tree's nodes that its mask names.

        kv_len (batch,), q_start (batch + 1,), q_off (batch,) and page_table (batch, width) int32. scale: 1 / sqrt(D)
        unless given. max_kv: the longest length to expect (the table's width unless given). Without a workspace one
        that ``workspace`` makes for the call's own bounds is allocated on the stream for this call."""
        T = q.shape[0]
        B = kv_len.shape[0]
        plain = self._plain
        qp, qt, qh = self._heads(q, "q", T, self.Hq)
        f32 = out.dtype is self._f32
        outp = plain(out, "out", self._f32 if f32 else self._f16, (T, self.Hq, self.D))
        lsep = 0 if lse is None else plain(lse, "lse", self._f32, (T, self.Hq))
        tp, ts, W = self._table(page_table, B)
        if max_kv is None:
            max_kv = max(1, W * self.page_tokens)
        handle = self._stream(stream)
        if workspace is None:
            import torch
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self.device)):
                workspace = self.workspace(B, max_q, max_kv)
        else:
            self._bytes(workspace)
        args = _pack_attend(B, max_q, T, qp, qt, qh,
                            0 if q_start is None else plain(q_start, "q_start", self._i32, (B + 1,)),
                            plain(kv_len, "kv_len", self._i32, (B,)),
                            0 if q_off is None else plain(q_off, "q_off", self._i32, (B,)),
                            tp, ts, W, bool(causal), max_kv, self.D ** -0.5 if scale is None else scale, f32, outp, lsep)
        if tree is None:
            rc = self._lib.kvc_attend(self._h, self._pages(pages), args, workspace.data_ptr(), workspace.numel(), handle)
        else:
            words = tree.shape[-1]
            rc = self._lib.kvc_attend_tree(self._h, self._pages(pages), args, plain(tree, "tree", self._i64, (T, words)),
                                           words, workspace.data_ptr(), workspace.numel(), handle)
        if rc != OK:
            self._raise(rc, "kvc_attend" if tree is None else "kvc_attend_tree")

    def tree(self, parent, q_start, kv_len, page_table, max_q: int, mask, positions=None, slots=None, total_len=None,
             stream=None):
        """kvc_tree: lays out a step's drafted tokens. parent (T,) int32, q_start (batch + 1,), kv_len (batch,) and
        page_table (batch, width) int32 give mask (T, words) int64, positions and slots (T,) int64 and total_len
        (batch,) int32. page_table may be None without slots."""
        T, B = parent.shape[0], kv_len.shape[0]
        plain, i32, i64 = self._plain, self._i32, self._i64
        words = mask.shape[-1]
        tp, ts, W = (0, 0, 0) if page_table is None else self._table(page_table, B)
        args = _pack_tree(B, max_q, T, plain(q_start, "q_start", i32, (B + 1,)), plain(kv_len, "kv_len", i32, (B,)),
                          plain(parent, "parent", i32, (T,)), tp, ts, W, words, plain(mask, "mask", i64, (T, words)),
                          0 if positions is None else plain(positions, "positions", i64, (T,)),
                          0 if slots is None else plain(slots, "slots", i64, (T,)),
                          0 if total_len is None else plain(total_len, "total_len", i32, (B,)))
        rc = self._lib.kvc_tree(self._h, args, self._stream(stream))
        if rc != OK:
            self._raise(rc, "kvc_tree")

    def verify_workspace(self, batch: int, vocab: int):
        """Workspace for every ``verify`` call within these bounds: one for each call that may run at the same time."""
        import torch
        n = _i64()
        rc = self._lib.kvc_verify_workspace(self._h, int(batch), int(vocab), ctypes.byref(n))
        if rc != OK:
            raise AgemmError(rc, f"kvc_verify_workspace: {status_string(rc)}")
        return torch.empty(max(16, n.value), dtype=torch.uint8, device=self.device)

    def verify(self, tokens, parent, q_start, p, u, path, count, next_token, max_q: int, q=None, max_children: int = 1,
               workspace=None, stream=None):
        """kvc_verify: the accepted path of each sequence's tree and the token that follows it.

        tokens (T,) int64, parent (T,) int32 and u (T,) float32, q_start (batch + 1,) int32; p and q (T, V) float32, the
        target's and the draft's probabilities after each node (q None: drafts are certain). path (T,) and count
        (batch,) int32 and next_token (batch,) int64 are written. max_children: the most children of a node to
        expect; drafts drawn in trees take up to ten times as long with the 1 of chains. Without a workspace one is allocated on the stream for this call."""
        T, B = parent.shape[0], count.shape[0]
        plain, i32, i64 = self._plain, self._i32, self._i64
        pp, ps, V = self._probabilities(p, "p", T)
        qp = qs = 0
        if q is not None:
            qp, qs, VQ = self._probabilities(q, "q", T)
            if VQ != V:
                raise ValueError(f"p and q must have the same vocabulary, got {V} and {VQ}")
        handle = self._stream(stream)
        if workspace is None:
            import torch
            with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(self.device)):
                workspace = self.verify_workspace(B, V)
        else:
            self._bytes(workspace)
        args = _pack_verify(B, max_q, T, plain(q_start, "q_start", i32, (B + 1,)), plain(parent, "parent", i32, (T,)),
                            plain(tokens, "tokens", i64, (T,)), pp, qp, ps, qs, V, plain(u, "u", self._f32, (T,)),
                            max_children, plain(path, "path", i32, (T,)), plain(count, "count", i32, (B,)),
                            plain(next_token, "next_token", i64, (B,)))
        rc = self._lib.kvc_verify(self._h, args, workspace.data_ptr(), workspace.numel(), handle)
        if rc != OK:
            self._raise(rc, "kvc_verify")

    def commit(self, pages, q_start, kv_len, path, count, page_table, max_q: int, new_len=None, stream=None):
        """kvc_commit: moves the accepted nodes of ``verify`` to their places, in the pages of one layer or a list of
        several with the same page table. new_len (batch,) int32: kv_len + count."""
        layers = pages if isinstance(pages, (list, tuple)) else (pages,)
        T, B = path.shape[0], kv_len.shape[0]
        plain, i32 = self._plain, self._i32
        tp, ts, W = self._table(page_table, B)
        args = _pack_commit(B, max_q, T, plain(q_start, "q_start", i32, (B + 1,)), plain(kv_len, "kv_len", i32, (B,)),
                            plain(path, "path", i32, (T,)), plain(count, "count", i32, (B,)), tp, ts, W,
                            0 if new_len is None else plain(new_len, "new_len", i32, (B,)))
        at = struct.pack(f"@{len(layers)}P", *[self._pages(p) for p in layers])
        rc = self._lib.kvc_commit(self._h, at, len(layers), args, self._stream(stream))
        if rc != OK:
            self._raise(rc, "kvc_commit")

    def read(self, pages, slots, k_out, v_out, stream=None):
        """kvc_read: the binary16 keys and values of the tokens in slots (T,) int64 into k_out and v_out (T, Hkv, D)."""
        T = slots.shape[0]
        shape = (T, self.Hkv, self.D)
        rc = self._lib.kvc_read(self._h, self._pages(pages), T, self._plain(slots, "slots", self._i64, (T,)),
                                self._plain(k_out, "k_out", self._f16, shape),
                                self._plain(v_out, "v_out", self._f16, shape), self._stream(stream))
        if rc != OK:
            self._raise(rc, "kvc_read")

    def check(self):
        """Raises AgemmError if a kernel met something it could not use (call after synchronising)."""
        self._raise(self._lib.kvc_check(self._h), "kvc_check")

    def close(self):
        if getattr(self, "_h", None):
            self._lib.kvc_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
