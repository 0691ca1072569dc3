// ds_kv4.cu -- host side of the 4-bit cache: argument checks and the entry
// points of ds_kv4.h that work on its tokens.
#include "ds_kv4.h"

#include "ds_host.h"
#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace {

using ds::fail;
using ds::fail_cuda;
using ds::kv4::Cache;

bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

int check_cache(const ds_kv4_cache_t *c, Cache *out)
{
    if (!c)
        return fail(DS_EINVAL, "cache is NULL");
    if (!dim_ok(c->head_dim))
        return fail(DS_EUNSUPPORTED, "head_dim = %d is not 64, 128 or 256", c->head_dim);
    if (c->n_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->max_seqs < 1 || c->max_pages < 1)
        return fail(DS_EINVAL,
                    "n_pages = %d, page_size = %d, kv_heads = %d, max_seqs = %d and max_pages = %d "
                    "must all be >= 1",
                    c->n_pages, c->page_size, c->kv_heads, c->max_seqs, c->max_pages);
    if ((long long)c->n_pages * c->page_size >= 1LL << 31)
        return fail(DS_EINVAL, "n_pages * page_size = %lld is not below 2^31",
                    (long long)c->n_pages * c->page_size);
    const long long page = (long long)c->kv_heads * c->page_size * ds::kv4::record_bytes(c->head_dim);
    if (c->page_stride % 16 != 0 || c->page_stride < page)
        return fail(DS_EINVAL, "page_stride = %lld is not a multiple of 16 of at least %lld bytes",
                    (long long)c->page_stride, page);
    if (c->table_stride < c->max_pages)
        return fail(DS_EINVAL, "table_stride = %lld is below max_pages = %d",
                    (long long)c->table_stride, c->max_pages);
    if (!c->pool || (uintptr_t)c->pool % 16 != 0)
        return fail(DS_EINVAL, "pool must be non-NULL and 16-byte aligned");
    if (!c->table)
        return fail(DS_EINVAL, "table must be non-NULL");
    out->pool = static_cast<unsigned char *>(c->pool);
    out->page_stride = c->page_stride;
    out->table = c->table;
    out->table_stride = c->table_stride;
    out->n_pages = c->n_pages;
    out->page_size = c->page_size;
    out->kv_heads = c->kv_heads;
    out->max_seqs = c->max_seqs;
    out->max_pages = c->max_pages;
    out->by_page.set(c->page_size);
    return DS_OK;
}

int check_dtype(int dtype)
{
    if (dtype != DS_FP32 && dtype != DS_BF16 && dtype != DS_FP16)
        return fail(DS_EUNSUPPORTED, "dtype %d is not DS_FP32 (0), DS_BF16 (1) or DS_FP16 (2)", dtype);
    return DS_OK;
}

int check_tokens(const Cache &c, const int32_t *seq, const int32_t *pos, int64_t tokens,
                 const void *k, const void *v)
{
    if (tokens < 0)
        return fail(DS_EINVAL, "tokens = %lld is negative", (long long)tokens);
    if (!ds::kv4::store_fits(c, tokens))
        return fail(DS_EUNSUPPORTED, "tokens = %lld are too many for one call", (long long)tokens);
    if (tokens > 0 && (!seq || !pos || !k || !v))
        return fail(DS_EINVAL, "seq, pos, k and v must be non-NULL when tokens > 0");
    return DS_OK;
}

int check_attention(const Cache &c, int batch, int queries, int heads, int k)
{
    if (batch < 0 || queries < 0 || heads < 1)
        return fail(DS_EINVAL, "batch = %d, queries = %d must be >= 0 and heads = %d >= 1", batch,
                    queries, heads);
    if (heads % c.kv_heads != 0)
        return fail(DS_EINVAL, "heads = %d is not a multiple of kv_heads = %d", heads, c.kv_heads);
    if (k < 0)
        return fail(DS_EINVAL, "k = %d is negative", k);
    if ((long long)batch * queries >= 1LL << 31 || (long long)batch * queries * heads >= 1LL << 31)
        return fail(DS_EUNSUPPORTED, "batch * queries * heads = %d * %d * %d is not below 2^31",
                    batch, queries, heads);
    return DS_OK;
}

}  // namespace

extern "C" {

int ds_kv4_record_bytes(int head_dim)
{
    if (!dim_ok(head_dim))
        return fail(DS_EUNSUPPORTED, "head_dim = %d is not 64, 128 or 256", head_dim);
    return ds::kv4::record_bytes(head_dim);
}

int ds_kv4_append(const ds_kv4_cache_t *cache, const int32_t *seq, const int32_t *pos,
                  int64_t tokens, int dtype, const void *k, const int64_t *k_stride, const void *v,
                  const int64_t *v_stride, void *stream)
{
    ds::g_detail[0] = '\0';
    Cache c;
    int rc = check_cache(cache, &c);
    if (rc == DS_OK)
        rc = check_dtype(dtype);
    if (rc == DS_OK)
        rc = check_tokens(c, seq, pos, tokens, k, v);
    if (rc != DS_OK)
        return rc;
    if (!k_stride || !v_stride)
        return fail(DS_EINVAL, "k_stride and v_stride must be non-NULL");
    if (tokens == 0)
        return DS_OK;
    const size_t size = dtype == DS_FP32 ? 4 : 2;
    if ((uintptr_t)k % size != 0 || (uintptr_t)v % size != 0)
        return fail(DS_EINVAL, "k and v must be aligned to their elements");
    const cudaError_t e = ds::kv4::launch_append(c, cache->head_dim, dtype, seq, pos, tokens, k,
                                                 k_stride, v, v_stride, (cudaStream_t)stream);
    return e == cudaSuccess ? DS_OK : fail_cuda(e, "ds_kv4_append");
}

int ds_kv4_read(const ds_kv4_cache_t *cache, const int32_t *seq, const int32_t *pos,
                int64_t tokens, int dtype, void *k, void *v, void *stream)
{
    ds::g_detail[0] = '\0';
    Cache c;
    int rc = check_cache(cache, &c);
    if (rc == DS_OK)
        rc = check_dtype(dtype);
    if (rc == DS_OK)
        rc = check_tokens(c, seq, pos, tokens, k, v);
    if (rc != DS_OK)
        return rc;
    if (tokens == 0)
        return DS_OK;
    if ((uintptr_t)k % 16 != 0 || (uintptr_t)v % 16 != 0)
        return fail(DS_EINVAL, "k and v must be 16-byte aligned");
    const cudaError_t e = ds::kv4::launch_read(c, cache->head_dim, dtype, seq, pos, tokens, k, v,
                                               (cudaStream_t)stream);
    return e == cudaSuccess ? DS_OK : fail_cuda(e, "ds_kv4_read");
}

int ds_kv4_attention_workspace(const ds_kv4_cache_t *cache, int batch, int queries, int heads,
                               int k, size_t *bytes)
{
    ds::g_detail[0] = '\0';
    Cache c;
    int rc = check_cache(cache, &c), dev = 0, sms = 0;
    if (rc == DS_OK)
        rc = check_attention(c, batch, queries, heads, k);
    if (rc != DS_OK)
        return rc;
    if (!bytes)
        return fail(DS_EINVAL, "bytes must be non-NULL");
    if ((rc = ds::current_device(&dev, &sms)) != DS_OK)
        return rc;
    ds::kv4::Attend a = {};
    a.batch = batch;
    a.queries = queries;
    a.heads = heads;
    a.k = k;
    *bytes = batch == 0 || queries == 0 ? 0 : ds::kv4::attention_workspace(c, cache->head_dim, a, sms);
    return DS_OK;
}

int ds_kv4_attention(const ds_kv4_cache_t *cache, const int32_t *lengths, const int32_t *seqs,
                     int batch, int queries, int heads, int dtype, const void *q,
                     const int64_t *q_stride, const int32_t *indices, int k, float scale, void *out,
                     float *lse, void *workspace, size_t workspace_bytes, void *stream)
{
    ds::g_detail[0] = '\0';
    Cache c;
    int rc = check_cache(cache, &c), dev = 0, sms = 0;
    if (rc == DS_OK)
        rc = check_attention(c, batch, queries, heads, k);
    if (rc != DS_OK)
        return rc;
    if (dtype != DS_BF16 && dtype != DS_FP16)
        return fail(DS_EUNSUPPORTED, "dtype %d is not DS_BF16 (1) or DS_FP16 (2)", dtype);
    if ((indices != nullptr) != (k > 0))
        return fail(DS_EINVAL, "indices need k >= 1, and k > 0 needs indices (k = %d)", k);
    if (!q_stride)
        return fail(DS_EINVAL, "q_stride must be non-NULL");
    if (batch == 0 || queries == 0)
        return DS_OK;
    if (!lengths || !q || !out)
        return fail(DS_EINVAL, "lengths, q and out must be non-NULL when batch and queries are > 0");
    if ((uintptr_t)q % 2 != 0 || (uintptr_t)out % 16 != 0)
        return fail(DS_EINVAL, "q must be aligned to its elements and out to 16 bytes");
    if ((rc = ds::current_device(&dev, &sms)) != DS_OK)
        return rc;
    ds::kv4::Attend a;
    a.lengths = lengths;
    a.seqs = seqs;
    a.indices = indices;
    a.q = q;
    a.q_batch = q_stride[0];
    a.q_query = q_stride[1];
    a.q_head = q_stride[2];
    a.out = out;
    a.lse = lse;
    a.partial = static_cast<float *>(workspace);
    a.scale = scale;
    a.batch = batch;
    a.queries = queries;
    a.heads = heads;
    a.k = k;
    a.bf16 = dtype == DS_BF16;
    const size_t need = ds::kv4::attention_workspace(c, cache->head_dim, a, sms);
    if (need > 0 && (!workspace || (uintptr_t)workspace % 16 != 0 || workspace_bytes < need))
        return fail(DS_EINVAL, "workspace must be 16-byte aligned and hold %zu bytes (%zu given)",
                    need, workspace_bytes);
    const cudaError_t e = ds::kv4::launch_attention(c, cache->head_dim, a, dev, sms,
                                                    (cudaStream_t)stream);
    return e == cudaSuccess ? DS_OK : fail_cuda(e, "ds_kv4_attention");
}

}  // extern "C"
