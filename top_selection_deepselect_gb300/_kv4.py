"""ctypes binding of include/ds_kv4.h -- the 4-bit paged cache that selected
tokens live in -- argument marshalling only, as in _binding.

The functions named like C entry points take the same arguments; the kv4_* and
pages_* functions take torch tensors, allocate outputs and workspaces with
torch and enqueue on the current stream.
"""
import ctypes
import math

from ._binding import DS_BF16, DS_FP16, DS_FP32, _check, load_library

KV4_ENTRY_POINTS = ["ds_kv4_record_bytes", "ds_kv4_append", "ds_kv4_read", "ds_kv4_attention",
                    "ds_kv4_attention_workspace", "ds_pages_copy", "ds_pages_reserve",
                    "ds_pages_fork", "ds_pages_free", "ds_pages_compact", "ds_pages_workspace"]


class ds_kv4_cache_t(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("page_stride", ctypes.c_int64),
                ("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64)] + [
        (name, ctypes.c_int32) for name in ("n_pages", "page_size", "kv_heads", "head_dim",
                                            "max_seqs", "max_pages")]


class ds_page_pool_t(ctypes.Structure):
    _fields_ = [("pool", ctypes.c_void_p), ("layer_stride", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64),
                ("layers", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


class ds_page_book_t(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("table_stride", ctypes.c_int64),
                ("lengths", ctypes.c_void_p), ("refs", ctypes.c_void_p),
                ("max_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int32)]


_strides2 = ctypes.c_int64 * 2
_strides3 = ctypes.c_int64 * 3
_typed = None


def _lib():
    global _typed
    if _typed is None:
        lib = load_library()
        vp, i32, i64, size = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
        cache, pool, book = (ctypes.POINTER(t) for t in (ds_kv4_cache_t, ds_page_pool_t,
                                                         ds_page_book_t))
        args = {
            "ds_kv4_record_bytes": [i32],
            "ds_kv4_append": [cache, vp, vp, i64, i32, vp, _strides2, vp, _strides2, vp],
            "ds_kv4_read": [cache, vp, vp, i64, i32, vp, vp, vp],
            "ds_kv4_attention": [cache, vp, vp, i32, i32, i32, i32, vp, _strides3, vp, i32,
                                 ctypes.c_float, vp, vp, vp, size, vp],
            "ds_kv4_attention_workspace": [cache, i32, i32, i32, i32, ctypes.POINTER(size)],
            "ds_pages_copy": [pool, vp, vp, i32, vp],
            "ds_pages_reserve": [book, vp, vp, i32, vp, vp, size, vp],
            "ds_pages_fork": [pool, book, vp, vp, i32, vp, vp, size, vp],
            "ds_pages_free": [book, vp, i32, vp],
            "ds_pages_compact": [pool, book, vp, vp, vp, size, vp],
            "ds_pages_workspace": [i32, i32],
        }
        for name, a in args.items():
            getattr(lib, name).argtypes = a
            getattr(lib, name).restype = size if name == "ds_pages_workspace" else i32
        _typed = lib
    return _typed


# ---- C entry points, same names and argument order ---------------------------
def ds_kv4_record_bytes(head_dim):
    r = _lib().ds_kv4_record_bytes(head_dim)
    if r < 0:
        _check(r, "ds_kv4_record_bytes")
    return r


def ds_kv4_append(cache, seq, pos, tokens, dtype, k, k_stride, v, v_stride, stream):
    return _check(_lib().ds_kv4_append(cache, seq, pos, tokens, dtype, k, _strides2(*k_stride), v,
                                       _strides2(*v_stride), stream), "ds_kv4_append")


def ds_kv4_read(cache, seq, pos, tokens, dtype, k, v, stream):
    return _check(_lib().ds_kv4_read(cache, seq, pos, tokens, dtype, k, v, stream), "ds_kv4_read")


def ds_kv4_attention(cache, lengths, seqs, batch, queries, heads, dtype, q, q_stride, indices, k,
                     scale, out, lse, workspace, workspace_bytes, stream):
    return _check(_lib().ds_kv4_attention(cache, lengths, seqs, batch, queries, heads, dtype, q,
                                          _strides3(*q_stride), indices, k, scale, out, lse,
                                          workspace, workspace_bytes, stream), "ds_kv4_attention")


def ds_kv4_attention_workspace(cache, batch, queries, heads, k):
    n = ctypes.c_size_t(0)
    _check(_lib().ds_kv4_attention_workspace(cache, batch, queries, heads, k, ctypes.byref(n)),
           "ds_kv4_attention_workspace")
    return n.value


def ds_pages_copy(pool, src, dst, n, stream):
    return _check(_lib().ds_pages_copy(pool, src, dst, n, stream), "ds_pages_copy")


def ds_pages_reserve(book, seqs, tokens, n, status, workspace, workspace_bytes, stream):
    return _check(_lib().ds_pages_reserve(book, seqs, tokens, n, status, workspace,
                                          workspace_bytes, stream), "ds_pages_reserve")


def ds_pages_fork(pool, book, src, dst, n, status, workspace, workspace_bytes, stream):
    return _check(_lib().ds_pages_fork(pool, book, src, dst, n, status, workspace,
                                       workspace_bytes, stream), "ds_pages_fork")


def ds_pages_free(book, seqs, n, stream):
    return _check(_lib().ds_pages_free(book, seqs, n, stream), "ds_pages_free")


def ds_pages_compact(pool, book, remap, status, workspace, workspace_bytes, stream):
    return _check(_lib().ds_pages_compact(pool, book, remap, status, workspace, workspace_bytes,
                                          stream), "ds_pages_compact")


def ds_pages_workspace(n_pages, n):
    return _lib().ds_pages_workspace(n_pages, n)


# ---- torch convenience wrappers ------------------------------------------------
def _torch():
    import torch
    return torch


def _code(dtype):
    t = _torch()
    code = {t.float32: DS_FP32, t.bfloat16: DS_BF16, t.float16: DS_FP16}.get(dtype)
    if code is None:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    return code


def _stream(x, stream):
    return (stream or _torch().cuda.current_stream(x.device)).cuda_stream


def _int32(name, t, device, shape=None):
    """Address of a contiguous CUDA int32 tensor."""
    if t.dtype != _torch().int32 or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, device))
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, shape, tuple(t.shape)))
    return t.data_ptr()


def _check_table(table, device):
    if (table.dtype != _torch().int32 or table.device != device or table.dim() != 2
            or table.stride(1) != 1 and table.shape[1] != 1):
        raise ValueError("table must be an int32 [max_seqs, max_pages] tensor on %s with unit "
                         "stride in the last dimension" % (device,))
    return max(table.stride(0), table.shape[1])


def kv4_record_bytes(head_dim):
    """Bytes of one token's record of one key/value head (head_dim 64, 128 or 256)."""
    return ds_kv4_record_bytes(head_dim)


def _cache(pool, table, head_dim):
    """Descriptor of a pool [n_pages, kv_heads, page_size, record bytes] (uint8) and its table."""
    if pool.dtype != _torch().uint8 or not pool.is_cuda or pool.dim() != 4:
        raise ValueError("pool must be a 4-D CUDA uint8 tensor [n_pages, kv_heads, page_size, "
                         "record bytes]")
    n_pages, kv_heads, page_size, rec = pool.shape
    if rec != ds_kv4_record_bytes(head_dim):
        raise ValueError("head_dim %d has records of %d bytes, the pool has %d"
                         % (head_dim, ds_kv4_record_bytes(head_dim), rec))
    if not pool[:1].is_contiguous():
        raise ValueError("each page of pool must be contiguous")
    stride = max(pool.stride(0), kv_heads * page_size * rec)
    return ds_kv4_cache_t(pool.data_ptr(), stride, table.data_ptr(),
                          _check_table(table, pool.device), n_pages, page_size, kv_heads, head_dim,
                          *table.shape)


def kv4_append(pool, table, seq, pos, k, v, stream=None):
    """Quantise tokens into the cache: token i goes to position pos[i] of sequence seq[i].

    k and v: [tokens, kv_heads, head_dim] float32, bfloat16 or float16, unit
    stride in the last dimension; seq and pos: int32 [tokens].  The pages must
    be in the table (pages_reserve); tokens without one are skipped.
    """
    if k.dim() != 3 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of one dtype")
    tokens, heads, dim = k.shape
    cache = _cache(pool, table, dim)
    if heads != cache.kv_heads:
        raise ValueError("k has %d heads, the pool %d" % (heads, cache.kv_heads))
    if k.device != pool.device or v.device != pool.device or k.stride(2) != 1 or v.stride(2) != 1:
        raise ValueError("k and v must be on the pool's device with unit stride in the last "
                         "dimension")
    ds_kv4_append(cache, _int32("seq", seq, pool.device, (tokens,)),
                  _int32("pos", pos, pool.device, (tokens,)), tokens, _code(k.dtype),
                  k.data_ptr(), k.stride()[:2], v.data_ptr(), v.stride()[:2],
                  _stream(pool, stream))


def kv4_read(pool, table, seq, pos, head_dim, dtype, k=None, v=None, stream=None):
    """Keys and values that the cache holds for tokens (seq[i], pos[i]).

    Returns (k, v), each [tokens, kv_heads, head_dim] of `dtype`; a token that
    is not there reads as zeros.
    """
    torch = _torch()
    cache = _cache(pool, table, head_dim)
    shape = (seq.numel(), cache.kv_heads, head_dim)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=pool.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=pool.device)
    for t in (k, v):
        if (tuple(t.shape) != shape or t.dtype != dtype or t.device != pool.device
                or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous %s tensors of %s" % (shape, dtype))
    ds_kv4_read(cache, _int32("seq", seq, pool.device, shape[:1]),
                _int32("pos", pos, pool.device, shape[:1]), shape[0], _code(dtype), k.data_ptr(),
                v.data_ptr(), _stream(pool, stream))
    return k, v


def kv4_attention(q, pool, table, lengths, indices=None, scale=None, seqs=None, out=None, lse=None,
                  workspace=None, stream=None):
    """Attention of q over the cache: over every token, or over the listed ones.

    q: [batch, queries, heads, head_dim] bfloat16 or float16, unit stride in
    the last dimension; entry b belongs to sequence seqs[b] (int32 [batch]), or
    b.  The queries are a sequence's newest tokens: query j of a sequence of L
    tokens (lengths, int32 [max_seqs]) sees those below L - queries + 1 + j.
    indices: int32 [batch, queries, k], positions to attend (as topk returns
    them for index scores; -1 and positions that the query does not see are
    left out).  scale defaults to 1 / sqrt(head_dim).  Returns (out, lse): out
    like q, lse float32 [batch, queries, heads]; a query that sees nothing gives
    0 and -inf.
    """
    torch = _torch()
    if q.dim() != 4 or q.device != pool.device or q.stride(3) != 1 and q.shape[3] != 1:
        raise ValueError("q must be [batch, queries, heads, head_dim] on the pool's device with "
                         "unit stride in the last dimension")
    batch, queries, heads, dim = q.shape
    cache = _cache(pool, table, dim)
    code = _code(q.dtype)
    device = pool.device
    at = _int32("lengths", lengths, device, (cache.max_seqs,))
    if seqs is None:
        if batch > cache.max_seqs:
            raise ValueError("batch = %d is above the table's %d sequences" % (batch, cache.max_seqs))
        seqs_at = None
    else:
        seqs_at = _int32("seqs", seqs, device, (batch,))
    k, list_at = 0, None
    if indices is not None:
        if indices.dim() != 3 or indices.shape[0] != batch or indices.shape[1] != queries:
            raise ValueError("indices must be [batch, queries, k]")
        k = indices.shape[2]
        list_at = _int32("indices", indices, device)
    if out is None:
        out = torch.empty((batch, queries, heads, dim), dtype=q.dtype, device=device)
    elif out.shape != q.shape or out.dtype != q.dtype or out.device != device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse is None:
        lse = torch.empty((batch, queries, heads), dtype=torch.float32, device=device)
    elif (lse.shape != q.shape[:3] or lse.dtype != torch.float32 or lse.device != device
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [batch, queries, heads] tensor")
    if indices is not None and k == 0:
        out.zero_()
        lse.fill_(-math.inf)
        return out, lse
    need = ds_kv4_attention_workspace(cache, batch, queries, heads, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    elif workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace has %d bytes, %d needed"
                         % (workspace.numel() * workspace.element_size(), need))
    ds_kv4_attention(cache, at, seqs_at, batch, queries, heads, code, q.data_ptr(), q.stride()[:3],
                     list_at, k, 1.0 / math.sqrt(dim) if scale is None else scale, out.data_ptr(),
                     lse.data_ptr(), workspace.data_ptr(),
                     workspace.numel() * workspace.element_size(), _stream(pool, stream))
    return out, lse


def _pool(pool):
    """Descriptor of a pool [layers, n_pages, ...] of pages of any content."""
    if not pool.is_cuda or pool.dim() < 3:
        raise ValueError("pool must be a CUDA tensor [layers, n_pages, ...]")
    layers, n_pages = pool.shape[:2]
    if not pool[:1, :1].is_contiguous():
        raise ValueError("each page of pool must be contiguous")
    size = pool.element_size()
    page = pool[0, 0].numel() * size
    return ds_page_pool_t(pool.data_ptr(), pool.stride(0) * size, max(pool.stride(1) * size, page),
                          page, layers, n_pages)


def _book(table, lengths, refs, page_size):
    device = table.device
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    stride = _check_table(table, device)
    return ds_page_book_t(
        table.data_ptr(), stride,
        None if lengths is None else _int32("lengths", lengths, device, (table.shape[0],)),
        _int32("refs", refs, device), *table.shape, page_size, refs.numel())


def _work(device, n_pages, n, workspace, status):
    torch = _torch()
    need = ds_pages_workspace(n_pages, n)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if status is None:
        status = torch.empty(2, dtype=torch.int32, device=device)
    else:
        _int32("status", status, device, (2,))
    return workspace, workspace.numel() * workspace.element_size(), status


def pages_copy(pool, src, dst, stream=None):
    """Page dst[i] of pool [layers, n_pages, ...] := page src[i], in every layer (int32 lists)."""
    n = src.numel()
    ds_pages_copy(_pool(pool), _int32("src", src, pool.device, (n,)),
                  _int32("dst", dst, pool.device, (n,)), n, _stream(pool, stream))


def pages_reserve(table, lengths, refs, seqs, tokens, page_size, workspace=None, status=None,
                  stream=None):
    """Sequence seqs[i] grows by tokens[i] tokens: lengths go up, missing pages are taken.

    All or nothing.  Returns status, int32 [2]: pages short (nothing changed
    when above 0), pages taken.
    """
    n = seqs.numel()
    book = _book(table, lengths, refs, page_size)
    workspace, size, status = _work(table.device, book.n_pages, n, workspace, status)
    ds_pages_reserve(book, _int32("seqs", seqs, table.device, (n,)),
                     _int32("tokens", tokens, table.device, (n,)), n, status.data_ptr(),
                     workspace.data_ptr(), size, _stream(table, stream))
    return status


def pages_fork(pool, table, lengths, refs, src, dst, workspace=None, status=None, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] that shares its full pages.

    pool: [layers, n_pages, kv_heads, page_size, record bytes].  All or nothing;
    returns status as pages_reserve does.
    """
    n = src.numel()
    if pool.dim() != 5:
        raise ValueError("pool must be [layers, n_pages, kv_heads, page_size, record bytes]")
    book = _book(table, lengths, refs, pool.shape[3])
    workspace, size, status = _work(table.device, book.n_pages, n, workspace, status)
    ds_pages_fork(_pool(pool), book, _int32("src", src, table.device, (n,)),
                  _int32("dst", dst, table.device, (n,)), n, status.data_ptr(),
                  workspace.data_ptr(), size, _stream(pool, stream))
    return status


def pages_free(table, lengths, refs, seqs, page_size, stream=None):
    """The sequences seqs[i] end: their pages' refs go down, their rows become -1."""
    n = seqs.numel()
    ds_pages_free(_book(table, lengths, refs, page_size),
                  _int32("seqs", seqs, table.device, (n,)), n, _stream(table, stream))


def pages_compact(pool, table, refs, workspace=None, remap=None, status=None, stream=None):
    """The live pages move to the front of pool [layers, n_pages, ...]; table and refs follow.

    Returns (remap int32 [n_pages]: new number of each page or -1, status int32
    [2]: live pages, pages moved).
    """
    torch = _torch()
    book = _book(table, None, refs, 1)
    if remap is None:
        remap = torch.empty(book.n_pages, dtype=torch.int32, device=table.device)
    workspace, size, status = _work(table.device, book.n_pages, 0, workspace, status)
    ds_pages_compact(_pool(pool), book, _int32("remap", remap, table.device, (book.n_pages,)),
                     status.data_ptr(), workspace.data_ptr(), size, _stream(pool, stream))
    return remap, status
