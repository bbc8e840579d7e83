"""Binding of the quantised key/value cache and its attention (``hqq_kv_*`` of ``include/hqq.h``).

As in the package itself the functions only marshal arguments: pages, queries and outputs are
torch tensors, every step runs in the library's kernels on the given or the current HIP stream.
"""
from __future__ import annotations

import ctypes
import struct
from dataclasses import dataclass

import weight_only_quantization_amd as _pkg

HQQ_KV_F16, HQQ_KV_BF16 = 0, 1

_p, _i64, _i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int


class KvCacheArgs(ctypes.Structure):
    """hqq_kv_cache of include/hqq.h."""
    _fields_ = [("pages", _p), ("num_pages", _i64), ("num_kv_heads", _i32), ("head_dim", _i32), ("nbits", _i32),
                ("group_size", _i32), ("page_size", _i32)]


class KvWriteArgs(ctypes.Structure):
    """hqq_kv_write_args of include/hqq.h."""
    _fields_ = [("cache", KvCacheArgs), ("dtype", _i32), ("k", _p), ("v", _p), ("n", _i64), ("k_token_stride", _i64),
                ("k_head_stride", _i64), ("v_token_stride", _i64), ("v_head_stride", _i64), ("slots", _p),
                ("k_echo", _p), ("v_echo", _p), ("stream", _p)]


class KvReadArgs(ctypes.Structure):
    """hqq_kv_read_args of include/hqq.h."""
    _fields_ = [("cache", KvCacheArgs), ("dtype", _i32), ("n", _i64), ("slots", _p), ("k", _p), ("v", _p),
                ("stream", _p)]


class KvAttentionArgs(ctypes.Structure):
    """hqq_kv_attention_args of include/hqq.h."""
    _fields_ = [("cache", KvCacheArgs), ("dtype", _i32), ("q", _p), ("total_q", _i64), ("q_token_stride", _i64),
                ("q_head_stride", _i64), ("num_q_heads", _i32), ("num_seqs", _i64), ("cu_q", _p), ("max_q", _i64),
                ("page_table", _p), ("table_stride", _i64), ("table_cols", _i64), ("seq_lens", _p), ("max_len", _i64),
                ("causal", _i32), ("scale", ctypes.c_float), ("prefix_table", _p), ("prefix_len", _i64), ("out", _p),
                ("lse", _p), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t), ("stream", _p)]


# The same structures as packed bytes (native alignment; a nested hqq_kv_cache ends in 4 bytes of
# padding): a call is a few microseconds, and filling a ctypes.Structure field by field would be a
# good part of them.
_CACHE = "Pqiiiiixxxx"
_WRITE = struct.Struct("@" + _CACHE + "iPPqqqqqPPPP")
_READ = struct.Struct("@" + _CACHE + "iqPPPP")
_ATTENTION = struct.Struct("@" + _CACHE + "iPqqqiqPqPqqPqifPqPPPNP")
assert (_WRITE.size, _READ.size, _ATTENTION.size) == tuple(map(ctypes.sizeof, (KvWriteArgs, KvReadArgs, KvAttentionArgs)))

_fast = {}  # entry points that take packed bytes


def declare(lib):
    """Argument types of the entry points (called when the library is loaded)."""
    lib.hqq_kv_page_bytes.argtypes = [_i32] * 5
    lib.hqq_kv_page_bytes.restype = ctypes.c_size_t
    for name, args in (("hqq_kv_write", KvWriteArgs), ("hqq_kv_read", KvReadArgs),
                       ("hqq_kv_attention", KvAttentionArgs), ("hqq_kv_attention_shared", KvAttentionArgs),
                       ("hqq_kv_attention_workspace_bytes", KvAttentionArgs)):
        fn = getattr(lib, name)
        fn.argtypes = [ctypes.POINTER(args)]
        fn.restype = ctypes.c_size_t if name.endswith("bytes") else _i32
        _fast[name] = ctypes.CFUNCTYPE(fn.restype, ctypes.c_char_p)((name, lib))


def _entry(name):
    if not _fast:
        _pkg.load()
    return _fast[name]


@dataclass
class KVCache:
    """Cache of one layer: `pages` is a contiguous uint8 tensor of num_pages pages (first
    dimension), each of hqq_kv_page_bytes(...) bytes; token slots are page * page_size + offset."""
    pages: "object"
    num_kv_heads: int
    head_dim: int
    nbits: int = 4
    group_size: int = 64
    page_size: int = 64

    @property
    def num_pages(self) -> int:
        return self.pages.shape[0]

    def args(self):
        """The fields of hqq_kv_cache, checked."""
        t = self.pages
        fmt = (self.num_kv_heads, self.head_dim, self.nbits, self.group_size, self.page_size)
        need = _sizes.get(fmt)
        if need is None:
            need = _page_bytes(*fmt)
        shape = t.shape
        if t.dtype is not _torch().uint8:
            raise ValueError("pages must be torch.uint8, got %s" % t.dtype)
        if not (t.is_cuda and t.is_contiguous()):
            _pkg._placed(t, "pages")
        if need and (len(shape) < 2 or t.numel() != shape[0] * need):
            raise ValueError("pages must be [num_pages, ...] of %d bytes a page, got %s" % (need, tuple(shape)))
        return (t.data_ptr(), shape[0], *fmt)


_sizes = {}


def _page_bytes(*fmt) -> int:
    if fmt not in _sizes:
        _sizes[fmt] = _pkg.load().hqq_kv_page_bytes(*fmt)
    return _sizes[fmt]


_modules = {}
_codes = {}


def _torch():
    t = _modules.get("torch")
    if t is None:
        import torch as t
        _modules["torch"] = t
        _codes.update({t.float16: HQQ_KV_F16, t.bfloat16: HQQ_KV_BF16})
    return t


def _dtype_code(dtype) -> int:
    _torch()
    code = _codes.get(dtype)
    if code is None:
        raise ValueError("dtype must be torch.float16 or torch.bfloat16, got %s" % dtype)
    return code


def _strides(t, name, heads, dim):
    """Token and head strides of a [tokens, heads, dim] tensor (channels contiguous)."""
    shape = t.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError("%s must be [tokens, %d, %d], got %s" % (name, heads, dim, tuple(shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor" % name)
    token, head, channel = t.stride()
    if channel != 1 or token % 8 or head % 8 or t.data_ptr() % 16:
        raise ValueError("%s needs contiguous channels, strides that are multiples of 8 elements and 16-byte alignment "
                         "(got strides %s); pass %s.contiguous()" % (name, t.stride(), name))
    return token, head


def _indices(t, name, dtype, dim):
    """Checks the values of an index tensor (slots, lengths, offsets; its place last, by _there) and returns its shape."""
    if not isinstance(t, _torch().Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    shape = t.shape
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if len(shape) != dim:
        raise ValueError("%s must have %d dimension%s, got %s" % (name, dim, "" if dim == 1 else "s", tuple(shape)))
    return shape


def _there(t, name):
    if not (t.is_cuda and t.is_contiguous()):
        _pkg._placed(t, name)


def _stream(stream, t):
    """The given stream's handle, or the current one's of the tensor's device."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(t.get_device())


def _empty(stream, shape, dtype, near):
    """A new tensor on the device of `near`, on the stream the kernels run on (see _on)."""
    if stream is None:
        return near.new_empty(shape, dtype=dtype)
    with _pkg._on(stream):
        return near.new_empty(shape, dtype=dtype)


def _like(stream, t):
    """A new contiguous tensor of t's shape and type (torch.empty_like is the faster call where t is contiguous)."""
    if stream is None and t.is_contiguous():
        return _torch().empty_like(t)
    return _empty(stream, t.shape, t.dtype, t)


def hqq_kv_page_bytes(num_kv_heads: int, head_dim: int, nbits: int = 4, group_size: int = 64,
                      page_size: int = 64) -> int:
    """Bytes of one page of a cache, 0 for a format the library does not have."""
    return _page_bytes(num_kv_heads, head_dim, nbits, group_size, page_size)


def hqq_kv_cache(num_pages: int, num_kv_heads: int, head_dim: int, nbits: int = 4, group_size: int = 64,
                 page_size: int = 64, device="cuda") -> KVCache:
    """Allocates the pages of one layer's cache (contents undefined: a token is written before it is
    read)."""
    nbytes = _pkg.load().hqq_kv_page_bytes(num_kv_heads, head_dim, nbits, group_size, page_size)
    if nbytes == 0:
        raise _pkg.HQQError(_pkg.HQQ_ERR_UNSUPPORTED, _pkg.last_error())
    pages = _torch().empty((num_pages, nbytes), dtype=_torch().uint8, device=device)
    return KVCache(pages, num_kv_heads, head_dim, nbits, group_size, page_size)


def hqq_kv_write(cache: KVCache, k, v, slots, echo: bool = False, stream=None):
    """Quantises k, v [n, num_kv_heads, head_dim] (fp16 or bf16; token and head strides allowed) into
    the cache's `slots` (int64 [n], distinct; slots outside the cache are skipped).  With `echo`
    returns (k, v) as the values the cache now stands for, else None (rounded once: in fp16 the top of a group that
    reaches 65504 may be infinite)."""
    count, = _indices(slots, "slots", _torch().int64, 1)
    dtype, n = k.dtype, k.shape[0]
    if v.dtype is not dtype:
        raise ValueError("k and v must have one dtype, got %s and %s" % (dtype, v.dtype))
    code = _codes.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    if v.shape[0] != n or count != n:
        raise ValueError("k, v and slots must have the same number of tokens")
    heads, dim = cache.num_kv_heads, cache.head_dim
    kt, kh = _strides(k, "k", heads, dim)
    vt, vh = _strides(v, "v", heads, dim)
    _there(slots, "slots")
    out = None
    if echo:
        first = _like(stream, k)
        out = (first, _like(stream, first))
    status = _entry("hqq_kv_write")(_WRITE.pack(
        *cache.args(), code, k.data_ptr(), v.data_ptr(), n, kt, kh, vt, vh, slots.data_ptr(),
        out[0].data_ptr() if echo else 0, out[1].data_ptr() if echo else 0, _stream(stream, k)))
    if status:
        _pkg._check(status)
    return out


def hqq_kv_read(cache: KVCache, slots, dtype=None, out=None, stream=None):
    """Keys and values (k, v), each [n, num_kv_heads, head_dim] of `dtype` (fp16 by default), that the
    cache's `slots` (int64 [n]) stand for; zeros for a slot outside the cache.  `out` = (k, v) takes
    them instead of new tensors."""
    torch = _torch()
    shape = (*_indices(slots, "slots", torch.int64, 1), cache.num_kv_heads, cache.head_dim)
    _there(slots, "slots")
    if out is None:
        dtype = dtype or torch.float16
        code = _dtype_code(dtype)
        first = _empty(stream, shape, dtype, slots)
        out = (first, _like(stream, first))
    else:
        code = _dtype_code(out[0].dtype)
        for t, name in zip(out, ("k", "v")):
            _pkg._need(t, name, out[0].dtype, shape=shape)
    status = _entry("hqq_kv_read")(_READ.pack(*cache.args(), code, shape[0], slots.data_ptr(), out[0].data_ptr(),
                                              out[1].data_ptr(), _stream(stream, slots)))
    if status:
        _pkg._check(status)
    return out


def hqq_kv_attention(cache: KVCache, q, page_table, seq_lens, scale=None, cu_q=None, max_q=None, max_len=None,
                     causal: bool = True, out=None, return_lse: bool = False, workspace=None, stream=None, _prefix=None):
    """Attention of query tokens q [total_q, heads, head_dim] over their sequences' cached tokens.

    page_table int32 [num_seqs, pages] and seq_lens int32 [num_seqs] (cached tokens, the query tokens
    included) are device tensors; cu_q int32 [num_seqs + 1] gives each sequence's range of query tokens (at
    most max_q; equal shares without it).  max_len bounds seq_lens for the launch (the table's
    length by default; pass the true bound: up to 2048 keys take a shorter path).  One call's sequences run by the
    longest one's number of query tokens, so decode steps and prompts' chunks are better called apart.  scale
    defaults to head_dim ** -0.5.  Returns out [total_q, heads, head_dim], with return_lse also the fp32 log-sum-exp [total_q,
    heads].  A row that sees no key is 0 (-inf)."""
    torch = _torch()
    dtype, dim, shape = q.dtype, cache.head_dim, q.shape
    code = _codes.get(dtype)
    if code is None:
        code = _dtype_code(dtype)
    if len(shape) != 3 or shape[2] != dim:
        raise ValueError("q must be [total_q, heads, %d], got %s" % (dim, tuple(shape)))
    total_q, heads, _ = shape
    qt, qh = _strides(q, "q", heads, dim)
    lens, = _indices(seq_lens, "seq_lens", torch.int32, 1)
    seqs, cols = _indices(page_table, "page_table", torch.int32, 2)
    _there(seq_lens, "seq_lens")
    row, col = page_table.stride()
    if not page_table.is_cuda or (col != 1 and cols > 1):
        raise ValueError("page_table must be a CUDA (HIP) tensor [num_seqs, pages], each row contiguous")
    if lens != seqs:
        raise ValueError("seq_lens must be [num_seqs] = [%d], got [%d]" % (seqs, lens))
    if cu_q is not None:
        if _indices(cu_q, "cu_q", torch.int32, 1)[0] != seqs + 1:
            raise ValueError("cu_q must be [num_seqs + 1]")
        _there(cu_q, "cu_q")
        if max_q is None or max_q > total_q:
            max_q = total_q
    entry, prefix_at, prefix_len = "hqq_kv_attention", 0, 0
    if _prefix is not None:
        entry = "hqq_kv_attention_shared"
        table, prefix_len = _prefix
        if prefix_len:
            pages, = _indices(table, "prefix_table", torch.int32, 1)
            _there(table, "prefix_table")
            if prefix_len < 0 or pages * cache.page_size < prefix_len:
                raise ValueError("prefix_table holds %d pages, too few for %d tokens" % (pages, prefix_len))
            prefix_at = table.data_ptr()
    most = cols * cache.page_size
    if out is None:
        out = _like(stream, q)
    else:
        _pkg._need(out, "out", dtype, shape=shape)
    lse = _empty(stream, (total_q, heads), torch.float32, q) if return_lse else None
    handle = _stream(stream, q)
    head = (*cache.args(), code, q.data_ptr(), total_q, qt, qh, heads, seqs, 0 if cu_q is None else cu_q.data_ptr(),
            max_q or 0, page_table.data_ptr(), row, cols, seq_lens.data_ptr(),
            most if max_len is None or max_len > most else max_len, 1 if causal else 0,
            dim ** -0.5 if scale is None else scale, prefix_at, prefix_len, out.data_ptr(), 0 if lse is None else lse.data_ptr())
    at = need = 0
    if workspace is None:
        need = _entry("hqq_kv_attention_workspace_bytes")(_ATTENTION.pack(*head, 0, 0, handle))
        if need:
            workspace = _empty(stream, need, torch.uint8, q)
            at = workspace.data_ptr()
    else:
        _pkg._need(workspace, "workspace", torch.uint8)
        at, need = workspace.data_ptr(), workspace.numel()
    status = _entry(entry)(_ATTENTION.pack(*head, at, need, handle))
    if status:
        _pkg._check(status)
    return out if lse is None else (out, lse)


def hqq_kv_attention_shared(cache: KVCache, q, prefix_table, prefix_len: int, page_table, seq_lens, scale=None,
                            cu_q=None, max_q=None, max_len=None, causal: bool = True, out=None,
                            return_lse: bool = False, workspace=None, stream=None):
    """hqq_kv_attention for sequences that share their first prefix_len tokens, kept once on the pages
    prefix_table (int32, device): every row sees the whole prefix, then its own sequence's cached tokens
    (page_table, seq_lens: without the prefix).  The prefix is read once for all rows together."""
    return hqq_kv_attention(cache, q, page_table, seq_lens, scale, cu_q, max_q, max_len, causal, out, return_lse,
                            workspace, stream, (prefix_table, prefix_len))
