"""Trees of drafted tokens and the paged key/value cache: binding of
sv_tree_attention, sv_verify_tree and sv_cache_* (see ``include/specverify.h``
for the conventions: tree rows, page tables, what is refused).

A decode step with a tree of k nodes, one layer shown:

    cache_append(k_new, v_new, k_cache[l], v_cache[l], page_table, seq_len)
    out = tree_attention(q, k_cache[l], v_cache[l], page_table, seq_len, parents).out
    r = verify_tree(target_logits, draft_logits, tokens, parents, uniforms, T)
    new_len = cache_commit(r.path, r.accepted_len, k_cache, v_cache, page_table, seq_len)
    cache_resize(new_len + k + 1, page_table, page_count, page_refs, page_size=page)

Calls run on the current stream of the tensors' device and may be captured
into a graph: during a capture a call without a `workspace` argument gets one
of its own.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

from . import (SV_BF16, SV_DRAFT_LOGITS, SV_DRAFT_ONEHOT, SVError, _check_dev, _dtype_code, _ptr, _stream_handle,
               _torch, _workspace_bytes, load_library)

__all__ = ["tree_attention", "TreeAttention", "verify_tree", "TreeVerifier", "cache_append", "cache_commit",
           "cache_fork", "cache_resize", "SV_F16"]

SV_F16 = 2

_i32, _i64 = ctypes.c_int32, ctypes.c_int64


class TreeAttentionDesc(ctypes.Structure):
    """sv_tree_attention_desc."""
    _fields_ = [("B", _i32), ("k", _i32), ("q_heads", _i32), ("kv_heads", _i32), ("head_dim", _i32),
                ("n_pages", _i32), ("page_size", _i32), ("max_pages", _i32), ("dtype", _i32),
                ("scale", ctypes.c_float), ("q_stride_b", _i64), ("q_stride_r", _i64), ("q_stride_h", _i64)]


class VerifyTreeDesc(ctypes.Structure):
    """sv_verify_tree_desc."""
    _fields_ = [("B", _i32), ("k", _i32), ("V", _i32), ("draft_rows", _i32), ("dtype", _i32), ("draft_kind", _i32),
                ("temperature", ctypes.c_float)]


class CacheDesc(ctypes.Structure):
    """sv_cache_desc."""
    _fields_ = [("n_seqs", _i32), ("n_pages", _i32), ("page_size", _i32), ("max_pages", _i32), ("n_layers", _i32),
                ("kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32)]


class CacheRows(ctypes.Structure):
    """sv_cache_rows."""
    _fields_ = [("t", _i32), ("k_stride_b", _i64), ("k_stride_t", _i64), ("k_stride_h", _i64),
                ("v_stride_b", _i64), ("v_stride_t", _i64), ("v_stride_h", _i64)]


def bind(lib) -> None:
    vp, sz, pt = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER
    for name, res, args in (
            ("sv_tree_attention_workspace_bytes", sz, [pt(TreeAttentionDesc)]),
            ("sv_tree_attention", ctypes.c_int, [pt(TreeAttentionDesc)] + [vp] * 9 + [sz, vp]),
            ("sv_verify_tree_workspace_bytes", sz, [pt(VerifyTreeDesc)]),
            ("sv_verify_tree", ctypes.c_int, [pt(VerifyTreeDesc)] + [vp] * 9 + [sz, vp]),
            ("sv_cache_append", ctypes.c_int, [pt(CacheDesc), pt(CacheRows)] + [vp] * 8),
            ("sv_cache_commit", ctypes.c_int, [pt(CacheDesc), _i32] + [vp] * 8),
            ("sv_cache_fork_workspace_bytes", sz, [pt(CacheDesc), _i32]),
            ("sv_cache_fork", ctypes.c_int, [pt(CacheDesc), _i32] + [vp] * 10 + [sz, vp]),
            ("sv_cache_resize", ctypes.c_int, [pt(CacheDesc)] + [vp] * 6)):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


class _Pool:
    """Workspaces by (device, stream), grown on demand to at least twice the size:
    calls on one stream run in order and share one, calls on others may overlap.
    An outgrown buffer is kept, as work on a stream that torch does not know may
    still use it.
    `zero`: the entry point wants its workspace zero-filled once."""

    def __init__(self, zero: bool):
        self._make = "zeros" if zero else "empty"
        self._buf, self._old = {}, []

    def new(self, device, nbytes: int):
        torch = _torch()
        return getattr(torch, self._make)(nbytes, dtype=torch.uint8, device=device)

    def get(self, device, nbytes: int, stream: int):
        buf = self._buf.get((device, stream))
        if buf is None or buf.numel() < nbytes:
            if buf is not None:
                self._old.append(buf)
                nbytes = max(nbytes, 2 * buf.numel())
            buf = self._buf[(device, stream)] = self.new(device, nbytes)
            if self._make == "zeros" and stream != _stream_of(device, None):
                _torch().cuda.current_stream(device).synchronize()  # the zeros are there before the other stream looks
        return buf


_WS_TREE = _Pool(zero=True)    # sv_verify_tree: zero-filled once, left ready by every call
_WS_PLAIN = _Pool(zero=False)  # the others: needs no clearing


def _workspace(pool, device, nbytes: int, given=None, own: bool = False, stream: Optional[int] = None):
    """The caller's workspace, checked, or one of the pool's; a buffer of its own
    for a prepared call (`own`) and while a graph is captured, so that two graphs
    never share one."""
    if given is not None:
        if given.device != device or not given.is_contiguous():
            raise ValueError("workspace must be contiguous and on %s" % device)
        if given.numel() * given.element_size() < nbytes:
            raise ValueError("workspace too small: need %d bytes" % nbytes)
        return given
    if device.type != "cuda" and not own:
        raise ValueError("tensors must be on a HIP device, got %s" % device)
    if own or _torch().cuda.is_current_stream_capturing():
        return pool.new(device, nbytes)
    return pool.get(device, nbytes, _stream_of(device, stream))


_HERE = contextlib.nullcontext()
_raw_stream = None


def _stream_of(device, stream):
    """The given stream, or the device's current one (by torch's raw query where
    it has one: half the time of building a Stream object)."""
    global _raw_stream
    if stream is not None:
        return stream
    if _raw_stream is None:
        raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = _stream_handle if raw is None else lambda d: raw(
            _torch().cuda.current_device() if d.index is None else d.index)
    return _raw_stream(device)


def _on(device):
    """Makes `device` the current one (the library launches on the current
    device).  Host tensors end here: their addresses must not reach a kernel."""
    torch = _torch()
    if device.type != "cuda":
        raise ValueError("tensors must be on a HIP device, got %s" % device)
    if device.index is None or device.index == torch.cuda.current_device():
        return _HERE
    return torch.cuda.device(device)


class _Plans(dict):
    """Checked descriptors by the call's signature (shapes, strides, types,
    devices): a call like an earlier one is not checked again.  Nothing of the
    tensors themselves is kept."""

    def keep(self, key, plan):
        if len(self) >= 256:
            self.clear()
        self[key] = plan
        return plan


def _sig(*tensors):
    """What the checks of a call look at."""
    return tuple(None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors)


_APPENDS, _COMMITS, _FORKS, _RESIZES = _Plans(), _Plans(), _Plans(), _Plans()


def _cache_dtype(t) -> int:
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return SV_BF16
    if t.dtype == torch.float16:
        return SV_F16
    raise TypeError("the cache must be torch.bfloat16 or torch.float16, got %s" % t.dtype)


def _rows_strides(name, t):
    if t.dim() != 4:
        raise ValueError("%s must be 4-dimensional (sequence, row, head, head_dim)" % name)
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError("%s: the head dimension must be contiguous" % name)
    # a dimension of one element may carry any stride, and is never stepped over
    return [s if n > 1 else 0 for s, n in zip(t.stride()[:3], t.shape[:3])]


def _check_cache(k_cache, v_cache, layers: bool):
    want = 5 if layers else 4
    if k_cache.dim() != want:
        raise ValueError("k_cache must be %s[pages][kv_heads][page_size][head_dim]" % ("[layers]" if layers else ""))
    _check_dev("k_cache", k_cache, k_cache.device)
    _check_dev("v_cache", v_cache, k_cache.device, k_cache.dtype, tuple(k_cache.shape))
    return _cache_dtype(k_cache)


def _cache_desc(n_seqs, max_pages, k_cache, layers: bool):
    shape = [int(n) for n in k_cache.shape]
    n_layers = shape[0] if layers else 1
    n_pages, heads, page, dim = shape[-4:]
    return CacheDesc(n_seqs, n_pages, page, max_pages, n_layers, heads, dim, _cache_dtype(k_cache))


def _table_shape(page_table, device):
    torch = _torch()
    if page_table.dim() != 2:
        raise ValueError("page_table must be [sequences][max_pages]")
    _check_dev("page_table", page_table, device, torch.int32)
    return int(page_table.shape[0]), int(page_table.shape[1])


class TreeAttentionOutput(NamedTuple):
    out: "object"
    lse: "object"


class TreeAttention:
    """A prepared sv_tree_attention call: descriptor, outputs and workspace built
    once.  The tensors are read at each call, so lengths, trees, pages and
    queries may change in place between calls.  Without `workspace` the call owns
    one; calls that never overlap in time (the layers of a model on one stream)
    may pass a common one."""

    def __init__(self, q, k_cache, v_cache, page_table, seq_len, parents=None, *, scale: Optional[float] = None,
                 return_lse: bool = False, out=None, workspace=None, _pooled: bool = False):
        torch = _torch()
        lib = load_library()
        device = q.device
        strides = _rows_strides("q", q)
        B, rows, heads, dim = (int(n) for n in q.shape)
        k = rows - 1
        code = _check_cache(k_cache, v_cache, layers=False)
        if k_cache.device != device:
            raise ValueError("k_cache is on %s, expected %s" % (k_cache.device, device))
        if q.dtype != k_cache.dtype:
            raise TypeError("q must be %s, got %s" % (k_cache.dtype, q.dtype))
        if int(k_cache.shape[3]) != dim:
            raise ValueError("the cache has head_dim %d, q %d" % (k_cache.shape[3], dim))
        n, max_pages = _table_shape(page_table, device)
        if n != B:
            raise ValueError("page_table has %d rows, expected %d" % (n, B))
        _check_dev("seq_len", seq_len, device, torch.int32, (B,))
        if parents is None:
            if k != 0:
                raise ValueError("parents are required for a tree with draft nodes")
        else:
            _check_dev("parents", parents, device, torch.int32, (B, k))
        self.desc = TreeAttentionDesc(B, k, heads, int(k_cache.shape[1]), dim, int(k_cache.shape[0]),
                                      int(k_cache.shape[2]), max_pages, code,
                                      float(dim ** -0.5 if scale is None else scale), *strides)
        nbytes = _workspace_bytes(lib, lib.sv_tree_attention_workspace_bytes, lib.sv_tree_attention, self.desc,
                                  [None] * 9 + [0, None], "sv_tree_attention")
        workspace = _workspace(_WS_PLAIN, device, nbytes, workspace, own=not _pooled)
        if out is None:
            out = torch.empty((B, rows, heads, dim), dtype=q.dtype, device=device)
        else:
            _check_dev("out", out, device, q.dtype, (B, rows, heads, dim))
        self.out = out
        self.lse = torch.empty((B, rows, heads), dtype=torch.float32, device=device) if return_lse else None
        self._keep = (q, k_cache, v_cache, page_table, seq_len, parents, workspace)
        self._lib, self._device = lib, device
        self._args = (ctypes.byref(self.desc), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(page_table),
                      _ptr(seq_len), _ptr(parents) if k else None, _ptr(self.out), _ptr(self.lse), _ptr(workspace),
                      workspace.numel() * workspace.element_size())

    def __call__(self, stream: Optional[int] = None) -> TreeAttentionOutput:
        with _on(self._device):
            st = self._lib.sv_tree_attention(*self._args, _stream_of(self._device, stream))
        if st:
            raise SVError(st, "sv_tree_attention", self._lib)
        return TreeAttentionOutput(self.out, self.lse)


def tree_attention(q, k_cache, v_cache, page_table, seq_len, parents=None, *, scale: Optional[float] = None,
                   return_lse: bool = False, out=None, workspace=None) -> TreeAttentionOutput:
    """sv_tree_attention on torch tensors of one HIP device.

    q [B][k+1][q_heads][head_dim] bf16/fp16, any strides that are multiples of
    8 with a contiguous head dimension; k_cache, v_cache [pages][kv_heads]
    [page_size][head_dim] of q's type, contiguous, the tree's rows appended;
    page_table [B][max_pages], seq_len [B], parents [B][k] int32 (None when k is
    0); scale 1/sqrt(head_dim) by default.  Returns (out, lse or None), out
    contiguous of q's shape (given or not, it must not overlap q).
    """
    return TreeAttention(q, k_cache, v_cache, page_table, seq_len, parents, scale=scale, return_lse=return_lse,
                         out=out, workspace=workspace, _pooled=True)()


class TreeVerifyOutput(NamedTuple):
    accepted_len: "object"
    out_tokens: "object"
    path: "object"


class TreeVerifier:
    """A prepared sv_verify_tree call (see :class:`TreeAttention`).  A `workspace`
    passed in must have been zero-filled once and serve sv_verify_tree alone."""

    def __init__(self, target, draft, draft_tokens, parents, uniforms, temperature: float, *, onehot: bool = False,
                 workspace=None, _pooled: bool = False):
        torch = _torch()
        lib = load_library()
        if target.dim() != 3:
            raise ValueError("target must be [B][k+1][V]")
        B, rows, V = (int(n) for n in target.shape)
        k = rows - 1
        device = target.device
        code = _dtype_code(target)
        _check_dev("target", target, device)
        greedy = float(temperature) == 0.0
        draft_rows = 0
        if onehot or greedy:
            draft = None
        else:
            if draft is None:
                raise ValueError("draft logits are required unless onehot or temperature == 0")
            if draft.dim() != 3:
                raise ValueError("draft must be [B][draft_rows][V]")
            draft_rows = int(draft.shape[1])
            _check_dev("draft", draft, device, target.dtype, (B, draft_rows, V))
        _check_dev("draft_tokens", draft_tokens, device, torch.int32, (B, k))
        _check_dev("parents", parents, device, torch.int32, (B, k))
        if greedy:
            uniforms = None
        else:
            if uniforms is None:
                raise ValueError("uniforms are required unless temperature == 0")
            _check_dev("uniforms", uniforms, device, torch.float32, (B, k + 1))
        self.desc = VerifyTreeDesc(B, k, V, draft_rows, code, SV_DRAFT_ONEHOT if onehot else SV_DRAFT_LOGITS,
                                   float(temperature))
        nbytes = _workspace_bytes(lib, lib.sv_verify_tree_workspace_bytes, lib.sv_verify_tree, self.desc,
                                  [None] * 9 + [0, None], "sv_verify_tree")
        workspace = _workspace(_WS_TREE, device, nbytes, workspace, own=not _pooled)
        self.accepted_len = torch.empty(B, dtype=torch.int32, device=device)
        self.out_tokens = torch.empty((B, k + 1), dtype=torch.int32, device=device)
        self.path = torch.empty((B, k), dtype=torch.int32, device=device)
        self._keep = (target, draft, draft_tokens, parents, uniforms, workspace)
        self._lib, self._device = lib, device
        self._args = (ctypes.byref(self.desc), _ptr(target), _ptr(draft), _ptr(draft_tokens), _ptr(parents),
                      _ptr(uniforms), _ptr(self.accepted_len), _ptr(self.out_tokens), _ptr(self.path),
                      _ptr(workspace), workspace.numel() * workspace.element_size())

    def __call__(self, stream: Optional[int] = None) -> TreeVerifyOutput:
        with _on(self._device):
            st = self._lib.sv_verify_tree(*self._args, _stream_of(self._device, stream))
        if st:
            raise SVError(st, "sv_verify_tree", self._lib)
        return TreeVerifyOutput(self.accepted_len, self.out_tokens, self.path)


def verify_tree(target, draft, draft_tokens, parents, uniforms, temperature: float, *, onehot: bool = False,
                workspace=None) -> TreeVerifyOutput:
    """sv_verify_tree on torch tensors (all on one HIP device, contiguous).

    target [B][k+1][V] bf16/fp32, row 0 after the root, row 1+i after node i;
    draft [B][draft_rows][V] of the same type, the rows that nodes with children
    were extended from (ignored when onehot or temperature == 0); draft_tokens,
    parents [B][k] int32; uniforms [B][k+1] float32 (ignored at temperature 0).
    Returns (accepted_len [B], out_tokens [B][k+1], path [B][k]).
    """
    return TreeVerifier(target, draft, draft_tokens, parents, uniforms, temperature, onehot=onehot,
                        workspace=workspace, _pooled=True)()


def _append_plan(k_new, v_new, k_cache, v_cache, page_table, seq_len, count):
    torch = _torch()
    device = k_cache.device
    _check_cache(k_cache, v_cache, layers=False)
    ks, vs = _rows_strides("k_new", k_new), _rows_strides("v_new", v_new)
    B, t = int(k_new.shape[0]), int(k_new.shape[1])
    want = (B, t, int(k_cache.shape[1]), int(k_cache.shape[3]))
    for name, x in (("k_new", k_new), ("v_new", v_new)):
        if x.device != device:
            raise ValueError("%s is on %s, expected %s" % (name, x.device, device))
        if x.dtype != k_cache.dtype:
            raise TypeError("%s must be %s, got %s" % (name, k_cache.dtype, x.dtype))
        if tuple(x.shape) != want:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(x.shape), want))
    n, max_pages = _table_shape(page_table, device)
    if n != B:
        raise ValueError("page_table has %d rows, expected %d" % (n, B))
    _check_dev("seq_len", seq_len, device, torch.int32, (B,))
    if count is not None:
        _check_dev("count", count, device, torch.int32, (B,))
    return _cache_desc(B, max_pages, k_cache, layers=False), CacheRows(t, *ks, *vs)


def cache_append(k_new, v_new, k_cache, v_cache, page_table, seq_len, *, count=None,
                 stream: Optional[int] = None) -> None:
    """sv_cache_append: rows j < count[b] of k_new, v_new [B][t][kv_heads]
    [head_dim] (strides multiples of 8, head dimension contiguous) to positions
    seq_len[b] + j of one layer's cache."""
    lib = load_library()
    device = k_cache.device
    key = _sig(k_new, v_new, k_cache, v_cache, page_table, seq_len, count)
    plan = _APPENDS.get(key)
    if plan is None:
        plan = _APPENDS.keep(key, _append_plan(k_new, v_new, k_cache, v_cache, page_table, seq_len, count))
    desc, rows = plan
    with _on(device):
        st = lib.sv_cache_append(ctypes.byref(desc), ctypes.byref(rows), _ptr(k_new), _ptr(v_new), _ptr(count),
                                 _ptr(page_table), _ptr(seq_len), _ptr(k_cache), _ptr(v_cache),
                                 _stream_of(device, stream))
    if st:
        raise SVError(st, "sv_cache_append", lib)


def _commit_plan(path, accepted_len, k_cache, v_cache, page_table, seq_len, new_len):
    torch = _torch()
    device = k_cache.device
    _check_cache(k_cache, v_cache, layers=True)
    n, max_pages = _table_shape(page_table, device)
    if path.dim() != 2:
        raise ValueError("path must be [B][k]")
    k = int(path.shape[1])
    _check_dev("path", path, device, torch.int32, (n, k))
    _check_dev("accepted_len", accepted_len, device, torch.int32, (n,))
    _check_dev("seq_len", seq_len, device, torch.int32, (n,))
    _check_dev("new_len", new_len, device, torch.int32, (n,))
    return _cache_desc(n, max_pages, k_cache, layers=True), k


def cache_commit(path, accepted_len, k_cache, v_cache, page_table, seq_len, *, new_len=None,
                 stream: Optional[int] = None):
    """sv_cache_commit: moves the accepted branch's rows (path [B][k], accepted_len
    [B] of verify_tree) in every layer of k_cache, v_cache [layers][pages]... and
    returns the new lengths (`new_len` if given; it must not be seq_len)."""
    lib = load_library()
    device = k_cache.device
    if new_len is None:
        new_len = _torch().empty_like(seq_len)
    key = _sig(path, accepted_len, k_cache, v_cache, page_table, seq_len, new_len)
    plan = _COMMITS.get(key)
    if plan is None:
        plan = _COMMITS.keep(key, _commit_plan(path, accepted_len, k_cache, v_cache, page_table, seq_len, new_len))
    desc, k = plan
    with _on(device):
        st = lib.sv_cache_commit(ctypes.byref(desc), k, _ptr(path), _ptr(accepted_len), _ptr(page_table),
                                 _ptr(seq_len), _ptr(new_len), _ptr(k_cache), _ptr(v_cache),
                                 _stream_of(device, stream))
    if st:
        raise SVError(st, "sv_cache_commit", lib)
    return new_len


def _fork_plan(lib, src, dst, k_cache, v_cache, page_table, page_count, page_refs, seq_len, status):
    torch = _torch()
    device = k_cache.device
    _check_cache(k_cache, v_cache, layers=True)
    m, max_pages = _table_shape(page_table, device)
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    n = int(src.shape[0])
    _check_dev("src", src, device, torch.int32, (n,))
    _check_dev("dst", dst, device, torch.int32, (n,))
    _check_dev("page_count", page_count, device, torch.int32, (m,))
    _check_dev("page_refs", page_refs, device, torch.int32, (int(k_cache.shape[1]),))
    _check_dev("seq_len", seq_len, device, torch.int32, (m,))
    _check_dev("status", status, device, torch.int32, (n,))
    desc = _cache_desc(m, max_pages, k_cache, layers=True)
    return desc, n, max(256, lib.sv_cache_fork_workspace_bytes(ctypes.byref(desc), n))


def cache_fork(src, dst, k_cache, v_cache, page_table, page_count, page_refs, seq_len, *, status=None,
               workspace=None, stream: Optional[int] = None):
    """sv_cache_fork: sequence dst[i] continues src[i] (whole pages shared, a begun
    one copied in every layer).  Returns status [n] int32 (1 done, 0 refused)."""
    lib = load_library()
    device = k_cache.device
    if status is None:
        status = _torch().empty_like(src)
    key = _sig(src, dst, k_cache, v_cache, page_table, page_count, page_refs, seq_len, status)
    plan = _FORKS.get(key)
    if plan is None:
        plan = _FORKS.keep(key, _fork_plan(lib, src, dst, k_cache, v_cache, page_table, page_count, page_refs,
                                           seq_len, status))
    desc, n, nbytes = plan
    workspace = _workspace(_WS_PLAIN, device, nbytes, workspace, stream=stream)
    with _on(device):
        st = lib.sv_cache_fork(ctypes.byref(desc), n, _ptr(src), _ptr(dst), _ptr(page_table), _ptr(page_count),
                               _ptr(page_refs), _ptr(seq_len), _ptr(k_cache), _ptr(v_cache), _ptr(status),
                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                               _stream_of(device, stream))
    if st:
        raise SVError(st, "sv_cache_fork", lib)
    return status


def _resize_plan(want_len, page_table, page_count, page_refs, status, page_size):
    torch = _torch()
    device = page_table.device
    m, max_pages = _table_shape(page_table, device)
    _check_dev("want_len", want_len, device, torch.int32, (m,))
    _check_dev("page_count", page_count, device, torch.int32, (m,))
    _check_dev("page_refs", page_refs, device, torch.int32)
    _check_dev("status", status, device, torch.int32, (m,))
    # the pages' contents are not touched: one head of eight stands for any shape
    return CacheDesc(m, int(page_refs.numel()), int(page_size), max_pages, 1, 1, 8, SV_BF16)


def cache_resize(want_len, page_table, page_count, page_refs, *, page_size: int, status=None,
                 stream: Optional[int] = None):
    """sv_cache_resize: gives every sequence the pages for want_len[b] positions
    (negative: as it is, 0: frees all).  Returns status [B] int32 (1 done, 0
    refused and unchanged)."""
    lib = load_library()
    device = page_table.device
    if status is None:
        status = _torch().empty_like(want_len)
    key = (_sig(want_len, page_table, page_count, page_refs, status), page_size)
    desc = _RESIZES.get(key)
    if desc is None:
        desc = _RESIZES.keep(key, _resize_plan(want_len, page_table, page_count, page_refs, status, page_size))
    with _on(device):
        st = lib.sv_cache_resize(ctypes.byref(desc), _ptr(want_len), _ptr(page_table), _ptr(page_count),
                                 _ptr(page_refs), _ptr(status), _stream_of(device, stream))
    if st:
        raise SVError(st, "sv_cache_resize", lib)
    return status
