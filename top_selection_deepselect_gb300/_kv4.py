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
# These run once a layer and step, around kernels of a few microseconds: what
# does not change (types, record sizes, workspace sizes) is looked up once.
_RECORD = {64: 80, 128: 144, 256: 288}
_torch_names = None


def _names():
    """(torch, int32, uint8, float32, dtype codes, raw stream of a device index)."""
    global _torch_names
    if _torch_names is None:
        import torch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            def raw(index):
                return torch.cuda.current_stream(index).cuda_stream
        _torch_names = (torch, torch.int32, torch.uint8, torch.float32,
                        {torch.float32: DS_FP32, torch.bfloat16: DS_BF16, torch.float16: DS_FP16}, raw)
    return _torch_names


def _code(dtype):
    code = _names()[4].get(dtype)
    if code is None:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    return code


def _stream(device, stream):
    return _names()[5](device.index) if stream is None else stream.cuda_stream


def _int32(name, t, device, n=None):
    """Address of a contiguous CUDA int32 tensor, of n entries in one dimension if given."""
    if t.dtype is not _names()[1] or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on %s" % (name, device))
    if n is not None and (t.dim() != 1 or t.shape[0] != n):
        raise ValueError("%s must have shape (%d,), got %s" % (name, n, tuple(t.shape)))
    return t.data_ptr()


def _table(table, device):
    """(address, row stride, rows, columns) of a page table."""
    if table.dtype is not _names()[1] or table.device != device or table.dim() != 2:
        raise ValueError("table must be an int32 [max_seqs, max_pages] tensor on %s" % (device,))
    rows, columns = table.shape
    stride, unit = table.stride()
    if unit != 1 and columns != 1:
        raise ValueError("table must have unit stride in the last dimension")
    return table.data_ptr(), stride if stride > columns else columns, rows, columns


def kv4_record_bytes(head_dim):
    """Bytes of one token's record of one key/value head (head_dim 64, 128 or 256)."""
    return ds_kv4_record_bytes(head_dim)


def _cache(pool, table, head_dim):
    """Descriptor of a pool [n_pages, kv_heads, page_size, record bytes] (uint8) and its table."""
    if pool.dtype is not _names()[2] or not pool.is_cuda or pool.dim() != 4:
        raise ValueError("pool must be a 4-D CUDA uint8 tensor [n_pages, kv_heads, page_size, "
                         "record bytes]")
    n_pages, kv_heads, page_size, rec = pool.shape
    if rec != _RECORD.get(head_dim):
        raise ValueError("head_dim %d has records of %d bytes, the pool has %d"
                         % (head_dim, ds_kv4_record_bytes(head_dim), rec))
    stride = pool.stride()
    page = kv_heads * page_size * rec
    if stride[1:] != (page_size * rec, rec, 1) and not pool[:1].is_contiguous():
        raise ValueError("each page of pool must be contiguous")
    at, row, rows, columns = _table(table, pool.device)
    return ds_kv4_cache_t(pool.data_ptr(), stride[0] if stride[0] > page else page, at, row, n_pages,
                          page_size, kv_heads, head_dim, rows, columns)


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
    if heads != pool.shape[1]:
        raise ValueError("k has %d heads, the pool %d" % (heads, pool.shape[1]))
    device = pool.device
    ks, vs = k.stride(), v.stride()
    if k.device != device or v.device != device or ks[2] != 1 or vs[2] != 1:
        raise ValueError("k and v must be on the pool's device with unit stride in the last "
                         "dimension")
    ds_kv4_append(cache, _int32("seq", seq, device, tokens), _int32("pos", pos, device, tokens),
                  tokens, _code(k.dtype), k.data_ptr(), ks[:2], v.data_ptr(), vs[:2],
                  _stream(device, stream))


def kv4_read(pool, table, seq, pos, head_dim, dtype, k=None, v=None, stream=None):
    """Keys and values that the cache holds for tokens (seq[i], pos[i]).

    Returns (k, v), each [tokens, kv_heads, head_dim] of `dtype`; a token that
    is not there reads as zeros.
    """
    cache = _cache(pool, table, head_dim)
    tokens, device = seq.numel(), pool.device
    shape = (tokens, pool.shape[1], head_dim)
    code = _code(dtype)
    given = [t for t in (k, v) if t is not None]
    for t in given:
        if (tuple(t.shape) != shape or t.dtype != dtype or t.device != device
                or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous %s tensors of %s" % (shape, dtype))
    if k is None:
        k = _names()[0].empty(shape, dtype=dtype, device=device)
    if v is None:
        v = _names()[0].empty(shape, dtype=dtype, device=device)
    ds_kv4_read(cache, _int32("seq", seq, device, tokens), _int32("pos", pos, device, tokens),
                tokens, code, k.data_ptr(), v.data_ptr(), _stream(device, stream))
    return k, v


_attention_bytes = {}


def _attention_workspace(cache, batch, queries, heads, k, device):
    """Workspace bytes, which depend on these sizes and the device alone."""
    key = (cache.head_dim, cache.kv_heads, queries, heads, k > 0, device.index)
    need = _attention_bytes.get(key)
    if need is None:
        if len(_attention_bytes) > 1000:
            _attention_bytes.clear()
        need = _attention_bytes[key] = ds_kv4_attention_workspace(cache, batch, queries, heads, k)
    return need


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
    torch, _, _, float32, codes, _ = _names()
    device = pool.device
    if q.dim() != 4 or q.device != device:
        raise ValueError("q must be [batch, queries, heads, head_dim] on the pool's device")
    shape, qs, dtype = q.shape, q.stride(), q.dtype
    batch, queries, heads, dim = shape
    if qs[3] != 1:
        raise ValueError("q must have unit stride in the last dimension")
    cache = _cache(pool, table, dim)
    code = codes.get(dtype)
    if code is None:
        raise TypeError("q must be bfloat16 or float16, got %s" % dtype)
    rows = table.shape[0]
    at = _int32("lengths", lengths, device, rows)
    seqs_at = list_at = None
    if seqs is not None:
        seqs_at = _int32("seqs", seqs, device, batch)
    elif batch > rows:
        raise ValueError("batch = %d is above the table's %d sequences" % (batch, rows))
    k = 0
    if indices is not None:
        if indices.dim() != 3 or indices.shape[0] != batch or indices.shape[1] != queries:
            raise ValueError("indices must be [batch, queries, k]")
        k = indices.shape[2]
        list_at = _int32("indices", indices, device)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=device)
    elif out.shape != shape or out.dtype != dtype or out.device != device or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse is None:
        lse = torch.empty(shape[:3], dtype=float32, device=device)
    elif (lse.shape != shape[:3] or lse.dtype != float32 or lse.device != device
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [batch, queries, heads] tensor")
    if indices is not None and k == 0:
        out.zero_()
        lse.fill_(-math.inf)
        return out, lse
    need = _attention_workspace(cache, batch, queries, heads, k, device)
    if workspace is None:
        workspace, size = torch.empty(need, dtype=torch.uint8, device=device), need
    else:
        size = workspace.numel() * workspace.element_size()
        if size < need or workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on %s with %d bytes, got %d"
                             % (device, need, size))
    ds_kv4_attention(cache, at, seqs_at, batch, queries, heads, code, q.data_ptr(), qs[:3], list_at,
                     k, 1.0 / math.sqrt(dim) if scale is None else scale, out.data_ptr(),
                     lse.data_ptr(), workspace.data_ptr(), size, _stream(device, stream))
    return out, lse


def _pool(pool):
    """Descriptor of a pool [layers, n_pages, ...] of pages of any content."""
    shape = pool.shape
    if not pool.is_cuda or len(shape) < 3:
        raise ValueError("pool must be a CUDA tensor [layers, n_pages, ...]")
    if not (pool.is_contiguous() or pool[:1, :1].is_contiguous()):
        raise ValueError("each page of pool must be contiguous")
    size = pool.element_size()
    page = math.prod(shape[2:]) * size
    layer, each = pool.stride()[:2]
    return ds_page_pool_t(pool.data_ptr(), layer * size, max(each * size, page), page, *shape[:2])


def _book(table, lengths, refs, page_size):
    device = table.device
    if not table.is_cuda:
        raise ValueError("table must be a CUDA tensor")
    at, stride, rows, columns = _table(table, device)
    return ds_page_book_t(at, stride,
                          None if lengths is None else _int32("lengths", lengths, device, rows),
                          _int32("refs", refs, device), rows, columns, page_size, refs.numel())


def _work(device, n_pages, n, workspace, status):
    """(workspace address, its bytes, status); ones that are not given are made."""
    torch = _names()[0]
    need = ds_pages_workspace(n_pages, n)
    if workspace is None:
        workspace, size = torch.empty(need, dtype=torch.uint8, device=device), need
    else:
        size = workspace.numel() * workspace.element_size()
        if workspace.device != device or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on %s" % (device,))
    if status is None:
        status = torch.empty(2, dtype=torch.int32, device=device)
    else:
        _int32("status", status, device, 2)
    return workspace, size, status


def pages_copy(pool, src, dst, stream=None):
    """Page dst[i] of pool [layers, n_pages, ...] := page src[i], in every layer (int32 lists)."""
    n, device = src.numel(), pool.device
    ds_pages_copy(_pool(pool), _int32("src", src, device, n), _int32("dst", dst, device, n), n,
                  _stream(device, stream))


def pages_reserve(table, lengths, refs, seqs, tokens, page_size, workspace=None, status=None,
                  stream=None):
    """Sequence seqs[i] grows by tokens[i] tokens: lengths go up, missing pages are taken.

    All or nothing.  Returns status, int32 [2]: pages short (nothing changed
    when above 0), pages taken.
    """
    n, device = seqs.numel(), table.device
    book = _book(table, lengths, refs, page_size)
    workspace, size, status = _work(device, book.n_pages, n, workspace, status)
    ds_pages_reserve(book, _int32("seqs", seqs, device, n), _int32("tokens", tokens, device, n), n,
                     status.data_ptr(), workspace.data_ptr(), size, _stream(device, stream))
    return status


def pages_fork(pool, table, lengths, refs, src, dst, workspace=None, status=None, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] that shares its full pages.

    pool: [layers, n_pages, kv_heads, page_size, record bytes].  All or nothing;
    returns status as pages_reserve does.
    """
    if pool.dim() != 5 or pool.device != table.device:
        raise ValueError("pool must be [layers, n_pages, kv_heads, page_size, record bytes] on the "
                         "table's device")
    n, device = src.numel(), table.device
    book = _book(table, lengths, refs, pool.shape[3])
    workspace, size, status = _work(device, book.n_pages, n, workspace, status)
    ds_pages_fork(_pool(pool), book, _int32("src", src, device, n), _int32("dst", dst, device, n), n,
                  status.data_ptr(), workspace.data_ptr(), size, _stream(device, stream))
    return status


def pages_free(table, lengths, refs, seqs, page_size, stream=None):
    """The sequences seqs[i] end: their pages' refs go down, their rows become -1."""
    n, device = seqs.numel(), table.device
    ds_pages_free(_book(table, lengths, refs, page_size), _int32("seqs", seqs, device, n), n,
                  _stream(device, stream))


def pages_compact(pool, table, refs, workspace=None, remap=None, status=None, stream=None):
    """The live pages move to the front of pool [layers, n_pages, ...]; table and refs follow.

    Returns (remap int32 [n_pages]: new number of each page or -1, status int32
    [2]: live pages, pages moved).
    """
    device = table.device
    if pool.device != device:
        raise ValueError("pool and table must be on one device")
    book = _book(table, None, refs, 1)
    n_pages = book.n_pages
    if remap is None:
        remap = _names()[0].empty(n_pages, dtype=_names()[1], device=device)
    workspace, size, status = _work(device, n_pages, 0, workspace, status)
    ds_pages_compact(_pool(pool), book, _int32("remap", remap, device, n_pages), status.data_ptr(),
                     workspace.data_ptr(), size, _stream(device, stream))
    return remap, status
