"""ctypes binding of include/ds_kv4.h -- the 4-bit paged cache that selected
tokens live in -- argument marshalling only, as in _binding.

The functions named like C entry points take the same arguments; the kv4_* and
pages_* functions take torch tensors, allocate outputs and workspaces with
torch and enqueue on the current stream of the tensors' device, which need not
be the current device.
"""
import ctypes
import math
import struct

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
# These run once a layer and step, around kernels of a few microseconds, so that
# their own time counts: types and sizes are looked up once, and descriptors are
# packed as bytes, which costs a quarter of filling a ctypes structure.
_RECORD = {64: 80, 128: 144, 256: 288}
_pack_cache = struct.Struct("@PqPq6i").pack     # ds_kv4_cache_t
_pack_pool = struct.Struct("@P3q2i").pack       # ds_page_pool_t
_pack_book = struct.Struct("@PqPP4i").pack      # ds_page_book_t
_pack_2 = struct.Struct("@2q").pack
_pack_3 = struct.Struct("@3q").pack


class _Torch:
    """What the wrappers need of torch and of the library, found at the first call."""
    ready = False

    def find(self):
        import torch
        self.torch, self.empty, self.empty_like = torch, torch.empty, torch.empty_like
        self.int32, self.uint8, self.float32 = torch.int32, torch.uint8, torch.float32
        self.codes = {torch.float32: DS_FP32, torch.bfloat16: DS_BF16, torch.float16: DS_FP16}
        self.raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda index: torch.cuda.current_stream(index).cuda_stream)
        self.on_stream = torch.cuda.stream
        self.current = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        self.on_device = torch.cuda.device
        lib = _lib()

        def bytes_for(name, at):
            """The function with byte strings in the places `at` of its structures."""
            f = lib[name]
            f.argtypes = [ctypes.c_char_p if i in at else a
                          for i, a in enumerate(getattr(lib, name).argtypes)]
            f.restype = getattr(lib, name).restype
            return f

        self.append = bytes_for("ds_kv4_append", (0, 6, 8))
        self.read = bytes_for("ds_kv4_read", (0,))
        self.attention = bytes_for("ds_kv4_attention", (0, 8))
        self.workspace = bytes_for("ds_kv4_attention_workspace", (0,))
        self.copy = bytes_for("ds_pages_copy", (0,))
        self.reserve = bytes_for("ds_pages_reserve", (0,))
        self.fork = bytes_for("ds_pages_fork", (0, 1))
        self.free = bytes_for("ds_pages_free", (0,))
        self.compact = bytes_for("ds_pages_compact", (0, 1))
        self.ready = True
        return self


_t = _Torch()

def _int32(name, x, index, n=None):
    """Address of a contiguous int32 tensor on device `index`, of n entries in one dimension if given."""
    if x.dtype is not _t.int32 or x.get_device() != index or not x.is_contiguous():
        raise ValueError("%s must be a contiguous int32 tensor on cuda:%d" % (name, index))
    if n is not None and x.shape != (n,):
        raise ValueError("%s must have shape (%d,), got %s" % (name, n, tuple(x.shape)))
    return x.data_ptr()


def _table(table, index):
    """(address, row stride, rows, columns) of a page table on device `index`."""
    if table.dtype is not _t.int32 or table.get_device() != index or table.dim() != 2:
        raise ValueError("table must be an int32 [max_seqs, max_pages] tensor on cuda:%d" % index)
    rows, columns = table.shape
    stride, unit = table.stride()
    if unit != 1 and columns != 1:
        raise ValueError("table must have unit stride in the last dimension")
    if stride < columns:
        if rows > 1:
            raise ValueError("rows of table must not overlap")
        stride = columns
    return table.data_ptr(), stride, rows, columns


def _space(name, x, index):
    """Bytes of a workspace that was passed in."""
    if x.get_device() != index or not x.is_contiguous():
        raise ValueError("%s must be contiguous on cuda:%d" % (name, index))
    return x.numel() * x.element_size()


def _cuda(name, x):
    """Index of a tensor's CUDA device."""
    index = x.get_device()
    if index < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    return index


def _elsewhere(t, index, stream, call, *args):
    """The result of call(*args) with `stream`, or else device `index`, made current.

    The library launches on the calling thread's current device, so that a call
    enters that of its tensors first."""
    if stream is None:
        with t.on_device(index):
            return call(*args)
    if stream.device_index != index:
        raise ValueError("stream belongs to cuda:%d, the tensors to cuda:%d" % (stream.device_index, index))
    with t.on_stream(stream):      # what is allocated belongs to that stream
        return call(*args)


def kv4_record_bytes(head_dim):
    """Bytes of one token's record of one key/value head (head_dim 64, 128 or 256)."""
    return ds_kv4_record_bytes(head_dim)


def _cache(pool, table, head_dim, index):
    """Descriptor of a pool [n_pages, kv_heads, page_size, record bytes] (uint8) and its table."""
    if pool.dtype is not _t.uint8 or pool.dim() != 4:
        raise ValueError("pool must be a 4-D CUDA uint8 tensor [n_pages, kv_heads, page_size, "
                         "record bytes]")
    n_pages, kv_heads, page_size, rec = pool.shape
    if rec != _RECORD.get(head_dim):
        raise ValueError("head_dim %d has records of %d bytes, the pool has %d"
                         % (head_dim, ds_kv4_record_bytes(head_dim), rec))
    each, head, token, unit = pool.stride()
    page = kv_heads * page_size * rec
    if (unit != 1 or token != rec or head != page_size * rec) and not pool[:1].is_contiguous():
        raise ValueError("each page of pool must be contiguous")
    if each < page:
        if n_pages > 1:
            raise ValueError("pages of pool must not overlap")
        each = page
    at, row, rows, columns = _table(table, index)
    return _pack_cache(pool.data_ptr(), each, at, row, n_pages, page_size, kv_heads, head_dim, rows,
                       columns)


def kv4_append(pool, table, seq, pos, k, v, stream=None):
    """Quantise tokens into the cache: token i goes to position pos[i] of sequence seq[i].

    k and v: [tokens, kv_heads, head_dim] float32, bfloat16 or float16, unit
    stride in the last dimension; seq and pos: int32 [tokens].  The pages must
    be in the table (pages_reserve); tokens without one are skipped.
    """
    t = _t if _t.ready else _t.find()
    index = _cuda("pool", pool)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, kv4_append, pool, table, seq, pos, k, v)
    shape, dtype = k.shape, k.dtype
    if len(shape) != 3 or shape != v.shape or dtype != v.dtype:
        raise ValueError("k and v must be [tokens, kv_heads, head_dim] of one dtype")
    tokens, heads, dim = shape
    cache = _cache(pool, table, dim, index)
    if heads != pool.shape[1]:
        raise ValueError("k has %d heads, the pool %d" % (heads, pool.shape[1]))
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError("k and v must be float32, bfloat16 or float16, got %s" % dtype)
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if k.get_device() != index or v.get_device() != index or k2 != 1 or v2 != 1:
        raise ValueError("k and v must be on the pool's device with unit stride in the last "
                         "dimension")
    status = t.append(cache, _int32("seq", seq, index, tokens), _int32("pos", pos, index, tokens),
                      tokens, code, k.data_ptr(), _pack_2(k0, k1), v.data_ptr(), _pack_2(v0, v1),
                      t.raw_stream(index))
    if status:
        _check(status, "ds_kv4_append")


def kv4_read(pool, table, seq, pos, head_dim, dtype, k=None, v=None, stream=None):
    """Keys and values that the cache holds for tokens (seq[i], pos[i]).

    Returns (k, v), each [tokens, kv_heads, head_dim] of `dtype`; a token that
    is not there reads as zeros.
    """
    t = _t if _t.ready else _t.find()
    index = _cuda("pool", pool)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, kv4_read, pool, table, seq, pos, head_dim, dtype, k, v)
    tokens = seq.numel()
    cache = _cache(pool, table, head_dim, index)
    shape = (tokens, pool.shape[1], head_dim)
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError("dtype must be float32, bfloat16 or float16, got %s" % dtype)
    for x in (k, v):
        if x is not None and (x.shape != shape or x.dtype != dtype or x.get_device() != index
                              or not x.is_contiguous()):
            raise ValueError("k and v must be contiguous %s tensors of %s" % (shape, dtype))
    if k is None:
        k = t.empty(shape, dtype=dtype, device=pool.device)
    if v is None:
        v = t.empty_like(k)
    status = t.read(cache, _int32("seq", seq, index, tokens), _int32("pos", pos, index, tokens),
                    tokens, code, k.data_ptr(), v.data_ptr(), t.raw_stream(index))
    if status:
        _check(status, "ds_kv4_read")
    return k, v


_attention_bytes = {}


def _attention_workspace(cache, batch, queries, heads, k, key):
    """Workspace bytes, which depend on the sizes in `key` and the device alone."""
    n = ctypes.c_size_t(0)
    _check(_t.workspace(cache, batch, queries, heads, k, ctypes.byref(n)),
           "ds_kv4_attention_workspace")
    if len(_attention_bytes) > 10000:
        _attention_bytes.clear()
    _attention_bytes[key] = n.value
    return n.value


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
    t = _t if _t.ready else _t.find()
    index = _cuda("pool", pool)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, kv4_attention,
                          q, pool, table, lengths, indices, scale, seqs, out, lse, workspace)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 4 or q.get_device() != index:
        raise ValueError("q must be [batch, queries, heads, head_dim] on the pool's device")
    batch, queries, heads, dim = shape
    q0, q1, q2, q3 = q.stride()
    if q3 != 1:
        raise ValueError("q must have unit stride in the last dimension")
    cache = _cache(pool, table, dim, index)
    code = t.codes.get(dtype)
    if code is None:
        raise TypeError("q must be bfloat16 or float16, got %s" % dtype)
    rows = table.shape[0]
    at = _int32("lengths", lengths, index, rows)
    seqs_at = list_at = None
    if seqs is not None:
        seqs_at = _int32("seqs", seqs, index, batch)
    elif batch > rows:
        raise ValueError("batch = %d is above the table's %d sequences" % (batch, rows))
    k = 0
    if indices is not None:
        if indices.dim() != 3 or indices.shape[0] != batch or indices.shape[1] != queries:
            raise ValueError("indices must be [batch, queries, k]")
        k = indices.shape[2]
        list_at = _int32("indices", indices, index)
    if out is None:
        out = t.empty(shape, dtype=dtype, device=q.device)
    elif out.shape != shape or out.dtype != dtype or out.get_device() != index or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of q's shape and dtype")
    if lse is None:
        lse = t.empty((batch, queries, heads), dtype=t.float32, device=q.device)
    elif (lse.shape != shape[:3] or lse.dtype != t.float32 or lse.get_device() != index
          or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 [batch, queries, heads] tensor")
    if indices is not None and k == 0:
        out.zero_()
        lse.fill_(-math.inf)
        return out, lse
    key = (index, shape, k, pool.shape, table.shape)
    size = _attention_bytes.get(key)
    if size is None:
        size = _attention_workspace(cache, batch, queries, heads, k, key)
    if workspace is None:
        if size:
            workspace = t.empty(size, dtype=t.uint8, device=q.device)
    else:
        given = _space("workspace", workspace, index)
        if given < size:
            raise ValueError("workspace has %d bytes, %d needed" % (given, size))
    status = t.attention(cache, at, seqs_at, batch, queries, heads, code, q.data_ptr(),
                         _pack_3(q0, q1, q2), list_at, k, dim ** -0.5 if scale is None else scale,
                         out.data_ptr(), lse.data_ptr(),
                         None if workspace is None else workspace.data_ptr(), size, t.raw_stream(index))
    if status:
        _check(status, "ds_kv4_attention")
    return out, lse


def _pool(pool, index):
    """Descriptor of a pool [layers, n_pages, ...] of pages of any content."""
    shape = pool.shape
    if len(shape) < 3 or pool.get_device() != index:
        raise ValueError("pool must be a tensor [layers, n_pages, ...] on cuda:%d" % index)
    if not (pool.is_contiguous() or pool[:1, :1].is_contiguous()):
        raise ValueError("each page of pool must be contiguous")
    size = pool.element_size()
    page = math.prod(shape[2:]) * size
    layer, each = pool.stride()[:2]
    layer, each = layer * size, each * size
    if each < page or layer < page:
        if each < page and shape[1] > 1 or layer < page and shape[0] > 1:
            raise ValueError("pages of pool must not overlap")
        each, layer = max(each, page), max(layer, page)
    return _pack_pool(pool.data_ptr(), layer, each, page, shape[0], shape[1])


def _book(table, lengths, refs, page_size, index):
    """Descriptor of the pages' bookkeeping."""
    at, stride, rows, columns = _table(table, index)
    return _pack_book(at, stride,
                      0 if lengths is None else _int32("lengths", lengths, index, rows),
                      _int32("refs", refs, index), rows, columns, page_size, refs.numel())


def _status(status, table, index):
    if status is None:
        return _t.empty(2, dtype=_t.int32, device=table.device)
    _int32("status", status, index, 2)
    return status


def _pages_bytes(n_pages, n):
    """What ds_pages_workspace answers, without the call."""
    return 4 * (2 * n_pages + 2 * n + 4)


def _work(t, table, index, need, workspace):
    """(workspace, its bytes): the one that was passed in, or memory of the current stream for this
    call alone."""
    if workspace is None:
        return t.empty(need, dtype=t.uint8, device=table.device), need
    return workspace, _space("workspace", workspace, index)


def pages_copy(pool, src, dst, stream=None):
    """Page dst[i] of pool [layers, n_pages, ...] := page src[i], in every layer (int32 lists)."""
    t = _t if _t.ready else _t.find()
    index = _cuda("pool", pool)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, pages_copy, pool, src, dst)
    n = src.numel()
    status = t.copy(_pool(pool, index), _int32("src", src, index, n), _int32("dst", dst, index, n), n,
                    t.raw_stream(index))
    if status:
        _check(status, "ds_pages_copy")


def pages_reserve(table, lengths, refs, seqs, tokens, page_size, workspace=None, status=None,
                  stream=None):
    """Sequence seqs[i] grows by tokens[i] tokens: lengths go up, missing pages are taken.

    All or nothing.  Returns status, int32 [2]: pages short (nothing changed
    when above 0), pages taken.
    """
    t = _t if _t.ready else _t.find()
    index = _cuda("table", table)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, pages_reserve,
                          table, lengths, refs, seqs, tokens, page_size, workspace, status)
    n = seqs.numel()
    book = _book(table, lengths, refs, page_size, index)
    status = _status(status, table, index)
    seqs_at, tokens_at = _int32("seqs", seqs, index, n), _int32("tokens", tokens, index, n)
    workspace, size = _work(t, table, index, _pages_bytes(refs.numel(), n), workspace)
    rc = t.reserve(book, seqs_at, tokens_at, n, status.data_ptr(), workspace.data_ptr(), size,
                   t.raw_stream(index))
    if rc:
        _check(rc, "ds_pages_reserve")
    return status


def pages_fork(pool, table, lengths, refs, src, dst, workspace=None, status=None, stream=None):
    """Sequence dst[i] becomes a copy of sequence src[i] that shares its full pages.

    pool: [layers, n_pages, kv_heads, page_size, record bytes].  All or nothing;
    returns status as pages_reserve does.
    """
    t = _t if _t.ready else _t.find()
    index = _cuda("table", table)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, pages_fork,
                          pool, table, lengths, refs, src, dst, workspace, status)
    if pool.dim() != 5:
        raise ValueError("pool must be [layers, n_pages, kv_heads, page_size, record bytes]")
    n = src.numel()
    book = _book(table, lengths, refs, pool.shape[3], index)
    at, status = _pool(pool, index), _status(status, table, index)
    src_at, dst_at = _int32("src", src, index, n), _int32("dst", dst, index, n)
    workspace, size = _work(t, table, index, _pages_bytes(refs.numel(), n), workspace)
    rc = t.fork(at, book, src_at, dst_at, n, status.data_ptr(), workspace.data_ptr(), size,
                t.raw_stream(index))
    if rc:
        _check(rc, "ds_pages_fork")
    return status


def pages_free(table, lengths, refs, seqs, page_size, stream=None):
    """The sequences seqs[i] end: their pages' refs go down, their rows become -1."""
    t = _t if _t.ready else _t.find()
    index = _cuda("table", table)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, pages_free, table, lengths, refs, seqs, page_size)
    n = seqs.numel()
    rc = t.free(_book(table, lengths, refs, page_size, index), _int32("seqs", seqs, index, n), n,
                t.raw_stream(index))
    if rc:
        _check(rc, "ds_pages_free")


def pages_compact(pool, table, refs, workspace=None, remap=None, status=None, stream=None):
    """The live pages move to the front of pool [layers, n_pages, ...]; table and refs follow.

    Returns (remap int32 [n_pages]: new number of each page or -1, status int32
    [2]: live pages, pages moved).
    """
    t = _t if _t.ready else _t.find()
    index = _cuda("table", table)
    if stream is not None or index != t.current():
        return _elsewhere(t, index, stream, pages_compact,
                          pool, table, refs, workspace, remap, status)
    n_pages = refs.numel()
    book = _book(table, None, refs, 1, index)
    if remap is None:
        remap = t.empty_like(refs)
    at, status = _pool(pool, index), _status(status, table, index)
    remap_at = _int32("remap", remap, index, n_pages)
    workspace, size = _work(t, table, index, _pages_bytes(n_pages, 0), workspace)
    rc = t.compact(at, book, remap_at, status.data_ptr(), workspace.data_ptr(), size,
                   t.raw_stream(index))
    if rc:
        _check(rc, "ds_pages_compact")
    return remap, status
