"""Binding of the quantised key/value cache and its attention (``hqq_kv_*`` of ``include/hqq.h``).

As in the package itself the functions only marshal arguments: pages, queries and outputs are
torch tensors, every step runs in the library's kernels on the given or the current HIP stream.
"""
from __future__ import annotations

import ctypes
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


def declare(lib):
    """Argument types of the entry points (called when the library is loaded)."""
    lib.hqq_kv_page_bytes.argtypes = [_i32] * 5
    lib.hqq_kv_page_bytes.restype = ctypes.c_size_t
    for name, args in (("hqq_kv_write", KvWriteArgs), ("hqq_kv_read", KvReadArgs),
                       ("hqq_kv_attention", KvAttentionArgs), ("hqq_kv_attention_shared", KvAttentionArgs)):
        getattr(lib, name).argtypes = [ctypes.POINTER(args)]
        getattr(lib, name).restype = _i32
    lib.hqq_kv_attention_workspace_bytes.argtypes = [ctypes.POINTER(KvAttentionArgs)]
    lib.hqq_kv_attention_workspace_bytes.restype = ctypes.c_size_t


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

    def args(self) -> KvCacheArgs:
        t = self.pages
        _pkg._need(t, "pages", _torch().uint8)
        need = _page_bytes(self.num_kv_heads, self.head_dim, self.nbits, self.group_size, self.page_size)
        if need and (t.dim() < 2 or t.numel() != t.shape[0] * need):
            raise ValueError("pages must be [num_pages, ...] of %d bytes a page, got %s" % (need, tuple(t.shape)))
        return KvCacheArgs(t.data_ptr(), t.shape[0], self.num_kv_heads, self.head_dim, self.nbits, self.group_size,
                           self.page_size)


_sizes = {}


def _page_bytes(*fmt) -> int:
    if fmt not in _sizes:
        _sizes[fmt] = _pkg.load().hqq_kv_page_bytes(*fmt)
    return _sizes[fmt]


def _torch():
    import torch
    return torch


_codes = {}


def _dtype_code(dtype) -> int:
    if not _codes:
        t = _torch()
        _codes.update({t.float16: HQQ_KV_F16, t.bfloat16: HQQ_KV_BF16})
    if dtype not in _codes:
        raise ValueError("dtype must be torch.float16 or torch.bfloat16, got %s" % dtype)
    return _codes[dtype]


def _strides(t, name, heads, dim):
    """Token and head strides of a [tokens, heads, dim] tensor (channels contiguous)."""
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError("%s must be [tokens, %d, %d], got %s" % (name, heads, dim, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor" % name)
    s = t.stride()
    if s[2] != 1 or s[0] % 8 or s[1] % 8 or t.data_ptr() % 16:
        raise ValueError("%s needs contiguous channels, strides that are multiples of 8 elements and 16-byte alignment "
                         "(got strides %s); pass %s.contiguous()" % (name, s, name))
    return s[0], s[1]


def _stream(stream):
    return (stream if stream is not None else _torch().cuda.current_stream()).cuda_stream


def hqq_kv_page_bytes(num_kv_heads: int, head_dim: int, nbits: int = 4, group_size: int = 64,
                      page_size: int = 64) -> int:
    """Bytes of one page of a cache, 0 for a format the library does not have."""
    return _page_bytes(num_kv_heads, head_dim, nbits, group_size, page_size)


def hqq_kv_cache(num_pages: int, num_kv_heads: int, head_dim: int, nbits: int = 4, group_size: int = 64,
                 page_size: int = 64, device="cuda") -> KVCache:
    """Allocates the pages of one layer's cache (contents undefined: a token is written before it is
    read)."""
    nbytes = _page_bytes(num_kv_heads, head_dim, nbits, group_size, page_size)
    if nbytes == 0:
        raise _pkg.HQQError(_pkg.HQQ_ERR_UNSUPPORTED, _pkg.last_error())
    pages = _torch().empty((num_pages, nbytes), dtype=_torch().uint8, device=device)
    return KVCache(pages, num_kv_heads, head_dim, nbits, group_size, page_size)


def hqq_kv_write(cache: KVCache, k, v, slots, echo: bool = False, stream=None):
    """Quantises k, v [n, num_kv_heads, head_dim] (fp16 or bf16; token and head strides allowed) into
    the cache's `slots` (int64 [n], distinct; slots outside the cache are skipped).  With `echo`
    returns (k, v) as the values the cache now stands for, else None."""
    torch = _torch()
    _pkg._need(slots, "slots", torch.int64, device=False)
    if v.dtype != k.dtype:
        raise ValueError("k and v must have one dtype, got %s and %s" % (k.dtype, v.dtype))
    code = _dtype_code(k.dtype)
    n = k.shape[0]
    if slots.dim() != 1 or slots.shape[0] != n or v.shape[0] != n:
        raise ValueError("k, v and slots must have the same number of tokens")
    kt, kh = _strides(k, "k", cache.num_kv_heads, cache.head_dim)
    vt, vh = _strides(v, "v", cache.num_kv_heads, cache.head_dim)
    _pkg._placed(slots, "slots")
    ke = ve = None
    if echo:
        with _pkg._on(stream):
            ke, ve = (torch.empty(k.shape, dtype=k.dtype, device=k.device) for _ in range(2))
    a = KvWriteArgs(cache.args(), code, k.data_ptr(), v.data_ptr(), n, kt, kh, vt, vh, slots.data_ptr(),
                    ke.data_ptr() if echo else None, ve.data_ptr() if echo else None, _stream(stream))
    _pkg._check(_pkg.load().hqq_kv_write(a))
    return (ke, ve) if echo else None


def hqq_kv_read(cache: KVCache, slots, dtype=None, out=None, stream=None):
    """Keys and values (k, v), each [n, num_kv_heads, head_dim] of `dtype` (fp16 by default), that the
    cache's `slots` (int64 [n]) stand for; zeros for a slot outside the cache.  `out` = (k, v) takes
    them instead of new tensors."""
    torch = _torch()
    _pkg._need(slots, "slots", torch.int64)
    if slots.dim() != 1:
        raise ValueError("slots must be [n]")
    shape = (slots.shape[0], cache.num_kv_heads, cache.head_dim)
    if out is None:
        code = _dtype_code(dtype or torch.float16)
        with _pkg._on(stream):
            out = tuple(torch.empty(shape, dtype=dtype or torch.float16, device=slots.device) for _ in range(2))
    else:
        code = _dtype_code(out[0].dtype)
        for t, name in zip(out, ("k", "v")):
            _pkg._need(t, name, out[0].dtype, shape=shape)
    a = KvReadArgs(cache.args(), code, slots.shape[0], slots.data_ptr(), out[0].data_ptr(), out[1].data_ptr(),
                   _stream(stream))
    _pkg._check(_pkg.load().hqq_kv_read(a))
    return out


def _attention(entry, cache, q, page_table, seq_lens, scale, cu_q, max_q, max_len, causal, prefix_table, prefix_len,
               out, return_lse, workspace, stream):
    torch = _torch()
    code = _dtype_code(q.dtype)
    if q.dim() != 3 or q.shape[2] != cache.head_dim:
        raise ValueError("q must be [total_q, heads, %d], got %s" % (cache.head_dim, tuple(q.shape)))
    total_q, heads = q.shape[0], q.shape[1]
    qt, qh = _strides(q, "q", heads, cache.head_dim)
    _pkg._need(seq_lens, "seq_lens", torch.int32)
    _pkg._need(page_table, "page_table", torch.int32, device=False)
    if not page_table.is_cuda or page_table.dim() != 2 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be a CUDA (HIP) tensor [num_seqs, pages], each row contiguous")
    seqs, cols = page_table.shape
    if seq_lens.dim() != 1 or seq_lens.shape[0] != seqs:
        raise ValueError("seq_lens must be [num_seqs] = [%d], got %s" % (seqs, tuple(seq_lens.shape)))
    if cu_q is not None:
        _pkg._need(cu_q, "cu_q", torch.int32)
        if cu_q.dim() != 1 or cu_q.shape[0] != seqs + 1:
            raise ValueError("cu_q must be [num_seqs + 1]")
        if max_q is None:
            max_q = total_q
    if prefix_len:
        _pkg._need(prefix_table, "prefix_table", torch.int32)
        if prefix_len < 0 or prefix_table.numel() * cache.page_size < prefix_len:
            raise ValueError("prefix_table holds %d pages, too few for %d tokens" % (prefix_table.numel(), prefix_len))
    if scale is None:
        scale = cache.head_dim ** -0.5
    lse = None
    with _pkg._on(stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            _pkg._need(out, "out", q.dtype, shape=q.shape)
        if return_lse:
            lse = torch.empty((total_q, heads), dtype=torch.float32, device=q.device)
        a = KvAttentionArgs(cache.args(), code, q.data_ptr(), total_q, qt, qh, heads, seqs,
                            None if cu_q is None else cu_q.data_ptr(), max_q or 0, page_table.data_ptr(),
                            max(page_table.stride(0), cols), cols, seq_lens.data_ptr(),
                            cols * cache.page_size if max_len is None else min(max_len, cols * cache.page_size),
                            1 if causal else 0, scale, prefix_table.data_ptr() if prefix_len else None, prefix_len,
                            out.data_ptr(), lse.data_ptr() if return_lse else None, None, 0, _stream(stream))
        lib = _pkg.load()
        need = lib.hqq_kv_attention_workspace_bytes(a)
        if need and workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    if workspace is not None:
        _pkg._need(workspace, "workspace", torch.uint8)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    _pkg._check(getattr(lib, entry)(a))
    return (out, lse) if return_lse else out


def hqq_kv_attention(cache: KVCache, q, page_table, seq_lens, scale=None, cu_q=None, max_q=None, max_len=None,
                     causal: bool = True, out=None, return_lse: bool = False, workspace=None, stream=None):
    """Attention of query tokens q [total_q, heads, head_dim] over their sequences' cached tokens.

    page_table int32 [num_seqs, pages] and seq_lens int32 [num_seqs] (cached tokens, the query tokens
    included) are device tensors; cu_q int32 [num_seqs + 1] gives each sequence's range of query tokens (at
    most max_q; equal shares without it).  max_len bounds seq_lens for the launch (the table's
    length by default: pass the true bound, the split of the keys goes by it).  scale defaults to
    head_dim ** -0.5.  Returns out [total_q, heads, head_dim], with return_lse also the fp32 log-sum-exp [total_q,
    heads].  A row that sees no key is 0 (-inf)."""
    return _attention("hqq_kv_attention", cache, q, page_table, seq_lens, scale, cu_q, max_q, max_len, causal, None, 0,
                      out, return_lse, workspace, stream)


def hqq_kv_attention_shared(cache: KVCache, q, prefix_table, prefix_len: int, page_table, seq_lens, scale=None,
                            cu_q=None, max_q=None, max_len=None, causal: bool = True, out=None,
                            return_lse: bool = False, workspace=None, stream=None):
    """hqq_kv_attention for sequences that share their first prefix_len tokens, kept once on the pages
    prefix_table (int32, device): every row sees the whole prefix, then its own sequence's cached tokens
    (page_table, seq_lens: without the prefix).  The prefix is read once for all rows together."""
    return _attention("hqq_kv_attention_shared", cache, q, page_table, seq_lens, scale, cu_q, max_q, max_len, causal,
                      prefix_table, prefix_len, out, return_lse, workspace, stream)
