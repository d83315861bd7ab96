"""The paged key/value cache of the verify cycle (include/ds_cache.h).

``ds_cache_append``, ``ds_paged_attention``, ``ds_cache_update`` and
``ds_cache_compact`` are the ctypes binding: they keep the C names, forward
device pointers, sizes and the current CUDA stream, and return the status code
(``check`` raises on it). ``KvPool`` describes a pool of pages; ``PagedCache``
owns a pool with its tables and issues the calls of a cycle. As everywhere in
the package, PyTorch tensors are device memory only and there is no fallback.
"""

import ctypes
import math
import struct

import torch

from . import _lib
from ._lib import DS_BF16, DS_F32, check  # noqa: F401

# Every symbol include/ds_cache.h declares.
EXPORTS = ("ds_cache_append", "ds_paged_attention_workspace_bytes", "ds_paged_attention",
           "ds_cache_update_workspace_bytes", "ds_cache_update", "ds_cache_compact_workspace_bytes",
           "ds_cache_compact")

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class PoolDesc(ctypes.Structure):
    _fields_ = [("dtype", _i32), ("n_layers", _i32), ("n_pages", _i32), ("page_size", _i32),
                ("n_kv_heads", _i32), ("head_dim", _i32), ("k", _vp), ("v", _vp),
                ("layer_stride", _i64), ("page_stride", _i64), ("token_stride", _i64),
                ("head_stride", _i64)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("layer", _i32), ("B", _i32), ("T", _i32), ("max_pages", _i32),
                ("k_new", _vp), ("v_new", _vp), ("k_token_stride", _i64), ("k_head_stride", _i64),
                ("v_token_stride", _i64), ("v_head_stride", _i64), ("q_start", _vp),
                ("block_table", _vp), ("kv_len", _vp), ("status", _vp)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("layer", _i32), ("B", _i32), ("T", _i32), ("max_pages", _i32),
                ("max_q", _i32), ("n_heads", _i32), ("causal", _i32), ("window", _i32),
                ("scale", ctypes.c_float), ("q", _vp), ("q_token_stride", _i64),
                ("q_head_stride", _i64), ("q_start", _vp), ("block_table", _vp), ("kv_len", _vp),
                ("out", _vp), ("out_token_stride", _i64), ("out_head_stride", _i64), ("lse", _vp),
                ("workspace", _vp), ("workspace_bytes", _sz), ("status", _vp)]


class UpdateArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("B", _i32), ("max_pages", _i32), ("block_table", _vp),
                ("kv_len", _vp), ("ref", _vp), ("parent", _vp), ("new_len", _vp), ("table_out", _vp),
                ("len_out", _vp), ("ref_out", _vp), ("workspace", _vp), ("workspace_bytes", _sz),
                ("status", _vp)]


class CompactArgs(ctypes.Structure):
    _fields_ = [("pool", PoolDesc), ("B", _i32), ("max_pages", _i32), ("block_table", _vp),
                ("ref", _vp), ("table_out", _vp), ("ref_out", _vp), ("page_map", _vp),
                ("n_used", _vp), ("workspace", _vp), ("workspace_bytes", _sz), ("status", _vp)]


# A call's arguments are packed as bytes, the pool's first (filling in a ctypes structure
# field by field takes a fifth of a small call).
_CODES = {_i32: "i", _i64: "q", _vp: "P", _sz: "N", ctypes.c_float: "f"}


def _packer(args):
    """struct.pack for an argument structure's fields after the pool, with C's alignment."""
    assert args._fields_[0] == ("pool", PoolDesc)
    s = struct.Struct("@" + "".join(_CODES[t] for _, t in args._fields_[1:]) + "0P")
    assert ctypes.sizeof(PoolDesc) % 8 == 0 and ctypes.sizeof(PoolDesc) + s.size == ctypes.sizeof(args)
    return s.pack


_pack_append, _pack_attention = _packer(AppendArgs), _packer(AttentionArgs)
_pack_update, _pack_compact = _packer(UpdateArgs), _packer(CompactArgs)

_bound = None
_entries = {}   # the calls, taking packed arguments


def load():
    """The library with the cache's entry points typed (loaded once)."""
    global _bound
    if _bound is None:
        lib = _lib.load()
        for name, args in (("ds_cache_append", AppendArgs), ("ds_paged_attention", AttentionArgs),
                           ("ds_cache_update", UpdateArgs), ("ds_cache_compact", CompactArgs)):
            getattr(lib, name).argtypes = [ctypes.POINTER(args), _vp]
            getattr(lib, name).restype = ctypes.c_int
            _entries[name] = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, _vp)((name, lib))
        for name, args in (("ds_paged_attention_workspace_bytes", [_i32, _i32]),
                           ("ds_cache_update_workspace_bytes", [_i32, _i32]),
                           ("ds_cache_compact_workspace_bytes", [_i32])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = _sz
        _bound = lib
    return _bound


def _entry(name):
    if _bound is None:
        load()
    return _entries[name]


def _words(t, name, device=None, n=None, _int32=torch.int32):
    """Device address of a contiguous int32 tensor on CUDA device `device` (of n elements, if given)."""
    if t.dtype is _int32 and t.get_device() == device and t.is_contiguous() and (n is None or t.numel() == n):
        return t.data_ptr()
    if t.dtype is not _int32:
        raise ValueError("%s must be int32" % name)
    _on_device(t, name, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must have %d elements" % (name, n))


def _on_device(t, name, device):
    if t.get_device() != device:
        raise ValueError("%s must be a CUDA tensor on the pool's device (cuda:%s)" % (name, device))


def _rows(t, name, pool, shape, heads=None):
    """Device address, token and head stride of a tensor [T, heads, head_dim] (of that
    `shape`) of the pool's dtype."""
    if t.dtype is not pool.dtype:
        raise ValueError("%s must have the pool's dtype" % name)
    if t.get_device() != pool.device_index:
        _on_device(t, name, pool.device_index)
    if len(shape) != 3 or shape[2] != pool.head_dim or (heads is not None and shape[1] != heads):
        raise ValueError("%s must be [T, heads, head_dim]" % name)
    ts, hs, one = t.stride()
    if one != 1:
        raise ValueError("%s: the last index must be contiguous" % name)
    # a stride that is never taken may be anything in torch: give the natural one
    if shape[1] == 1:
        hs = pool.head_dim
    if shape[0] <= 1:
        ts = shape[1] * pool.head_dim
    return t.data_ptr(), ts, hs


def _bytes(t, name, device):
    if t.get_device() != device:
        _on_device(t, name, device)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr(), t.nbytes


def _stream(stream, pool):
    """The stream's handle; the current one of the pool's device by default (asked for
    without building a Stream object, which takes as long as the launches). Launches go to
    the current device, which has to be the pool's."""
    if torch._C._cuda_getDevice() != pool.device_index:
        raise ValueError("the pool is on cuda:%d, the current device is cuda:%d" %
                         (pool.device_index, torch._C._cuda_getDevice()))
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(pool.device_index)
    return _lib._stream(stream)


class KvPool:
    """A pool of pages: K and V as tensors [n_layers, n_pages, page_size,
    n_kv_heads, head_dim] of equal strides with the last index contiguous. Any
    order of the others in memory will do (``x.transpose(2, 3)`` for heads
    outside tokens)."""

    def __init__(self, k, v):
        if k.dim() != 5 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride():
            raise ValueError("k and v must be [n_layers, n_pages, page_size, n_kv_heads, head_dim] of one "
                             "dtype and equal strides")
        if not (k.is_cuda and v.is_cuda) or k.device != v.device:
            raise ValueError("k and v must be CUDA tensors of one device")
        if k.stride(4) != 1:
            raise ValueError("the last index of k and v must be contiguous")
        self.k, self.v = k, v
        self.dtype = k.dtype
        self.device_index = k.device.index
        self.n_layers, self.n_pages, self.page_size, self.n_kv_heads, self.head_dim = k.shape
        st = list(k.stride())
        # a stride that is never taken may be anything in torch: give a valid one
        if self.n_kv_heads == 1:
            st[3] = self.head_dim
        if self.n_pages == 1:
            st[1] = self.page_size * self.n_kv_heads * self.head_dim
        self.desc = PoolDesc(_lib._dtype_code(k), self.n_layers, self.n_pages, self.page_size, self.n_kv_heads,
                             self.head_dim, k.data_ptr(), v.data_ptr(), st[0], st[1], st[2], st[3])
        self.packed = bytes(self.desc)


def ds_cache_append(pool, layer, k_new, v_new, q_start, block_table, kv_len, status, stream=None):
    """New keys and values [T, n_kv_heads, head_dim] into their pages."""
    B, M = block_table.shape
    dev = pool.device_index
    shape = k_new.shape
    k, kt, kh = _rows(k_new, "k_new", pool, shape, pool.n_kv_heads)
    v, vt, vh = _rows(v_new, "v_new", pool, v_new.shape, pool.n_kv_heads)
    if v_new.shape != shape:
        raise ValueError("k_new and v_new must have one shape")
    a = pool.packed + _pack_append(layer, B, shape[0], M, k, v, kt, kh, vt, vh,
                   _words(q_start, "q_start", dev, B + 1), _words(block_table, "block_table", dev),
                   _words(kv_len, "kv_len", dev, B), _words(status, "status", dev))
    return _entry("ds_cache_append")(a, _stream(stream, pool))


def ds_paged_attention_workspace_bytes(pool, n_heads):
    """Workspace of ds_paged_attention on this pool (the same for every batch; 0: not supported)."""
    if n_heads % pool.n_kv_heads != 0:
        return 0
    return load().ds_paged_attention_workspace_bytes(pool.desc.dtype, pool.head_dim)


def ds_paged_attention(pool, layer, q, q_start, max_q, block_table, kv_len, out, workspace, status, lse=None,
                       causal=True, window=0, scale=None, stream=None):
    """Attention of ragged rows q [T, n_heads, head_dim] over the cache; `scale`
    defaults to 1 / sqrt(head_dim). Writes out and, if given, lse [T, n_heads] float32."""
    B, M = block_table.shape
    dev = pool.device_index
    shape = q.shape
    qp, qt, qh = _rows(q, "q", pool, shape)
    T, H = shape[0], shape[1]
    op, ot, oh = _rows(out, "out", pool, out.shape, H)
    if out.shape[0] != T:
        raise ValueError("out must have q's shape")
    lp = 0
    if lse is not None:
        if lse.dtype is not torch.float32 or lse.get_device() != dev or not lse.is_contiguous() or lse.numel() != T * H:
            raise ValueError("lse must be a contiguous float32 tensor [T, n_heads] on the pool's device")
        lp = lse.data_ptr()
    wp, wn = _bytes(workspace, "workspace", dev)
    a = pool.packed + _pack_attention(layer, B, T, M, max_q, H, 1 if causal else 0, window,
                      1.0 / math.sqrt(pool.head_dim) if scale is None else scale, qp, qt, qh,
                      _words(q_start, "q_start", dev, B + 1), _words(block_table, "block_table", dev),
                      _words(kv_len, "kv_len", dev, B), op, ot, oh, lp, wp, wn, _words(status, "status", dev))
    return _entry("ds_paged_attention")(a, _stream(stream, pool))


def ds_cache_update_workspace_bytes(B, n_pages):
    return load().ds_cache_update_workspace_bytes(B, n_pages)


def ds_cache_update(pool, block_table, kv_len, ref, new_len, table_out, len_out, ref_out, workspace, status,
                    parent=None, stream=None):
    """Every request's next state (out of place): see include/ds_cache.h."""
    B, M = block_table.shape
    dev = pool.device_index
    N = pool.n_pages
    wp, wn = _bytes(workspace, "workspace", dev)
    a = pool.packed + _pack_update(B, M, _words(block_table, "block_table", dev), _words(kv_len, "kv_len", dev, B),
                   _words(ref, "ref", dev, N), 0 if parent is None else _words(parent, "parent", dev, B),
                   _words(new_len, "new_len", dev, B), _words(table_out, "table_out", dev, B * M),
                   _words(len_out, "len_out", dev, B), _words(ref_out, "ref_out", dev, N), wp, wn,
                   _words(status, "status", dev))
    return _entry("ds_cache_update")(a, _stream(stream, pool))


def ds_cache_compact_workspace_bytes(n_pages):
    return load().ds_cache_compact_workspace_bytes(n_pages)


def ds_cache_compact(pool, block_table, ref, table_out, ref_out, page_map, n_used, workspace, status, stream=None):
    """Held pages to the front of the pool (state out of place, pages in place)."""
    B, M = block_table.shape
    dev = pool.device_index
    N = pool.n_pages
    wp, wn = _bytes(workspace, "workspace", dev)
    a = pool.packed + _pack_compact(B, M, _words(block_table, "block_table", dev), _words(ref, "ref", dev, N),
                    _words(table_out, "table_out", dev, B * M), _words(ref_out, "ref_out", dev, N),
                    _words(page_map, "page_map", dev, N), _words(n_used, "n_used", dev, 1), wp, wn, _words(status, "status", dev))
    return _entry("ds_cache_compact")(a, _stream(stream, pool))


class PagedCache:
    """A pool with the state of B requests, as a serving loop keeps it.

    The state (block table, lengths, holders' counts) has two copies; `update`
    and `compact` write the one and make it current. Nothing synchronises; errors
    the device finds are in `status` (`check_status` reads it). The calls share the
    state and a workspace: what is issued on several streams the caller orders."""

    def __init__(self, n_layers, n_pages, page_size, n_kv_heads, head_dim, max_requests, max_len,
                 dtype=torch.bfloat16, device="cuda", heads_outside=False):
        shape = ((n_layers, n_pages, n_kv_heads, page_size, head_dim) if heads_outside
                 else (n_layers, n_pages, page_size, n_kv_heads, head_dim))
        k, v = (torch.empty(shape, dtype=dtype, device=device) for _ in range(2))
        if heads_outside:
            k, v = k.transpose(2, 3), v.transpose(2, 3)
        self.pool = KvPool(k, v)
        B, M = max_requests, -(-max_len // page_size)
        dev = k.device

        def state():
            return (torch.full((B, M), -1, dtype=torch.int32, device=dev),
                    torch.zeros(B, dtype=torch.int32, device=dev),
                    torch.zeros(n_pages, dtype=torch.int32, device=dev))

        self._now, self._next = state(), state()
        self.page_map = torch.empty(n_pages, dtype=torch.int32, device=dev)
        self.n_used = torch.empty(4, dtype=torch.int32, device=dev)[:1]
        self.status = torch.zeros(4, dtype=torch.int32, device=dev)
        n = max(ds_cache_update_workspace_bytes(B, n_pages), ds_cache_compact_workspace_bytes(n_pages),
                ds_paged_attention_workspace_bytes(self.pool, n_kv_heads))
        self.workspace = torch.empty(n, dtype=torch.uint8, device=dev)

    @property
    def block_table(self):
        return self._now[0]

    @property
    def kv_len(self):
        return self._now[1]

    @property
    def ref(self):
        return self._now[2]

    def update(self, new_len, parent=None, stream=None):
        """Lengths `new_len` [B] for all requests, continuing `parent` [B] (default: each itself)."""
        t, n, r = self._now
        check(ds_cache_update(self.pool, t, n, r, new_len, *self._next, self.workspace, self.status, parent=parent,
                              stream=stream), "ds_cache_update")
        self._now, self._next = self._next, self._now

    def append(self, layer, k_new, v_new, q_start, stream=None):
        check(ds_cache_append(self.pool, layer, k_new, v_new, q_start, self.block_table, self.kv_len, self.status,
                              stream=stream), "ds_cache_append")

    def attend(self, layer, q, q_start, max_q, out=None, lse=None, causal=True, window=0, scale=None, stream=None):
        if out is None:
            if stream is None:
                out = torch.empty_like(q)
            else:   # of that stream's memory: blocks freed on the current one may still be in use there
                with torch.cuda.stream(torch.cuda.ExternalStream(_lib._stream(stream).value or 0, q.device)):
                    out = torch.empty_like(q)
        check(ds_paged_attention(self.pool, layer, q, q_start, max_q, self.block_table, self.kv_len, out,
                                 self.workspace, self.status, lse=lse, causal=causal, window=window, scale=scale,
                                 stream=stream), "ds_paged_attention")
        return out

    def compact(self, stream=None):
        """Held pages to the front; `n_used` and `page_map` say where they are."""
        t, n, r = self._now
        t2, n2, r2 = self._next
        check(ds_cache_compact(self.pool, t, r, t2, r2, self.page_map, self.n_used, self.workspace, self.status,
                               stream=stream), "ds_cache_compact")
        self._now, self._next = (t2, n, r2), (t, n2, r)

    def reset_status(self):
        self.status.zero_()

    def check_status(self, stream=None):
        check(_lib.ds_check_status(self.status, stream), "device status")
