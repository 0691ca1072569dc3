"""DeepSelect top-k for GB300 (sm_103a).

The product is the C-ABI library libds_topk.so (include/ds_topk.h), built
from hand-written CUDA in csrc/.  This package is its thin Python binding:
the functions named like the C entry points marshal arguments and raise on a
non-zero status; `topk` wraps them for torch tensors.  The paged 4-bit cache
that selected tokens live in (include/ds_kv4.h) has kv4_append, kv4_read,
kv4_attention and pages_reserve / fork / free / compact / copy.  There is no CPU
fallback: without the compiled library every call raises.
"""
from ._binding import (DS_BF16, DS_ECUDA, DS_EINVAL, DS_EUNSUPPORTED, DS_FP16, DS_FP32, DS_OK,
                       DS_ORDER_IDENTITY, DS_ORDER_RANDOM, ENTRY_POINTS, DSError,
                       ds_last_error_detail, ds_strerror, ds_topk, ds_topk_ex, ds_topk_host,
                       ds_topk_host_async, ds_topk_long_row, ds_topk_long_row_noalloc,
                       ds_topk_long_row_workspace, ds_topk_max_k, ds_topk_plan,
                       ds_topk_stats_order, library_path, load_library, row_range, topk,
                       topk_long_row)
from ._build import build
from ._kv4 import (KV4_ENTRY_POINTS, ds_kv4_append, ds_kv4_attention, ds_kv4_attention_workspace,
                   ds_kv4_cache_t, ds_kv4_read, ds_kv4_record_bytes, ds_page_book_t,
                   ds_page_pool_t, ds_pages_compact, ds_pages_copy, ds_pages_fork, ds_pages_free,
                   ds_pages_reserve, ds_pages_workspace, kv4_append, kv4_attention, kv4_read,
                   kv4_record_bytes, pages_compact, pages_copy, pages_fork, pages_free,
                   pages_reserve)

__all__ = ["DS_BF16", "DS_ECUDA", "DS_EINVAL", "DS_EUNSUPPORTED", "DS_FP16", "DS_FP32", "DS_OK",
           "DS_ORDER_IDENTITY", "DS_ORDER_RANDOM", "ENTRY_POINTS", "DSError", "build",
           "ds_last_error_detail", "ds_strerror", "ds_topk", "ds_topk_ex", "ds_topk_host",
           "ds_topk_host_async", "ds_topk_long_row", "ds_topk_long_row_noalloc",
           "ds_topk_long_row_workspace", "ds_topk_max_k", "ds_topk_plan", "ds_topk_stats_order",
           "library_path", "load_library", "row_range", "topk", "topk_long_row",
           "KV4_ENTRY_POINTS", "ds_kv4_append", "ds_kv4_attention", "ds_kv4_attention_workspace",
           "ds_kv4_cache_t", "ds_kv4_read", "ds_kv4_record_bytes", "ds_page_book_t",
           "ds_page_pool_t", "ds_pages_compact", "ds_pages_copy", "ds_pages_fork", "ds_pages_free",
           "ds_pages_reserve", "ds_pages_workspace", "kv4_append", "kv4_attention", "kv4_read",
           "kv4_record_bytes", "pages_compact", "pages_copy", "pages_fork", "pages_free",
           "pages_reserve"]
