/*
 * ds_kv4.h -- C ABI of the key/value cache that the selected tokens live in:
 * a paged cache held in 4 bits, attention over all of its tokens or over the
 * tokens that a top-k call chose, and the moving of its pages.  Part of
 * libds_topk.so; status codes, dtypes and error texts are those of ds_topk.h.
 *
 * Records.  One token of one key/value head is a record of
 * ds_kv4_record_bytes(D) bytes (D: head dimension, 64, 128 or 256):
 *     D/2 bytes   key codes, two a byte
 *     D/2 bytes   value codes
 *     D/32 fp16   key scales, one for each group of 32 channels
 *     D/32 fp16   value scales
 *     zeros up to a multiple of 16 bytes
 * so 80 (72 used), 144 and 288 bytes.  A code u in 0..15 stands for
 * (u - 8) * scale.  Quantisation of a group x: scale = fp16(max|x| * r) with r
 * the fp32 number nearest to 1/7 and the product rounded to fp32 first, u = 8 +
 * clamp(rint(fp32(x / scale)), -7, 7), u = 8 where the scale is 0; a scale beyond
 * fp16 is 65504 (the codes clamp), and a group with a NaN or an infinity gets the
 * scale NaN, so that it reads back as NaN.
 * Order inside a record, for each stretch of W = min(D, 128) channels, with
 * n = W / 32 groups: the key's 32-bit words (eight channels, lowest channel
 * in the lowest bits) stand with word 4 i + t of the stretch at place
 * n t + i (t < 4), the value's 16-bit pieces (four channels) with piece
 * 8 i + g at place n g + i (g < 8): each lane of a warp then finds the
 * operands of its matrix instructions side by side.
 *
 * Pages.  The pool is n_pages pages of [kv_heads][page_size] records, any
 * page_size >= 1, n_pages * page_size < 2^31; a sequence's tokens
 * [i * page_size, (i + 1) * page_size) are in page table[seq][i].  Free
 * entries are -1.  The pages of several layers can share one table: a pool
 * of each layer, or one pool with a layer stride.
 *
 * Device-side conditions that cannot be reported synchronously never read or
 * write out of bounds: a length beyond max_pages * page_size is read as that,
 * a negative one as 0, and a token whose sequence, position or page is out of
 * range is not there (append skips it, read gives zeros, attention leaves it
 * out).
 *
 * Asynchrony: every function only enqueues work on `stream`, allocates
 * nothing and keeps nothing from call to call.  Argument errors are reported
 * before anything is enqueued.  A workspace must not be used by another call
 * until this one is done on its stream; nothing in it needs to be set.
 */
#ifndef DS_KV4_H
#define DS_KV4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cache: pool (device, 16-byte aligned) and page table (device). */
typedef struct {
    void *pool;            /* page p, head h, slot s at p * page_stride + (h * page_size + s) * record */
    int64_t page_stride;   /* bytes, a multiple of 16, at least a page */
    const int32_t *table;  /* [max_seqs][table_stride], max_pages entries a row */
    int64_t table_stride;  /* entries between rows, >= max_pages */
    int32_t n_pages;
    int32_t page_size;     /* tokens of a page */
    int32_t kv_heads;
    int32_t head_dim;      /* 64, 128 or 256 */
    int32_t max_seqs;
    int32_t max_pages;
} ds_kv4_cache_t;

/* Bytes of a record for this head dimension, or DS_EUNSUPPORTED. */
int ds_kv4_record_bytes(int head_dim);

/*
 * ds_kv4_append -- quantise `tokens` keys and values into the cache.
 *   seq, pos  device int32[tokens]: the sequence and the position in it of
 *             each token; distinct pairs (one that is given twice may end as a
 *             mixture of both); a token with seq outside [0, max_seqs) or pos
 *             outside its sequence's pages is skipped
 *   k, v      device [tokens][kv_heads][head_dim] of `dtype` (DS_FP32,
 *             DS_BF16 or DS_FP16), unit stride in the last dimension,
 *             k_stride / v_stride = {token stride, head stride} in elements
 */
int ds_kv4_append(const ds_kv4_cache_t *cache, const int32_t *seq, const int32_t *pos,
                  int64_t tokens, int dtype, const void *k, const int64_t *k_stride, const void *v,
                  const int64_t *v_stride, void *stream);

/*
 * ds_kv4_read -- the keys and values that the cache holds, the inverse of
 * ds_kv4_append: k and v are device [tokens][kv_heads][head_dim], contiguous;
 * a token that is not there reads as zeros.
 */
int ds_kv4_read(const ds_kv4_cache_t *cache, const int32_t *seq, const int32_t *pos,
                int64_t tokens, int dtype, void *k, void *v, void *stream);

/*
 * ds_kv4_attention -- softmax(scale * q K^T) V over the cache.
 *   batch     sequences attended; entry b is sequence seqs[b] (device
 *             int32[batch]), or b when seqs is NULL
 *   lengths   device int32[max_seqs]: tokens of each sequence, the newest
 *             `queries` of them those of the queries: query j of a sequence
 *             of L tokens sees the tokens below max(0, L - queries + 1 + j)
 *   heads     query heads, a multiple of kv_heads; head h reads key/value
 *             head h / (heads / kv_heads)
 *   dtype     of q and out: DS_BF16 or DS_FP16
 *   q         device, unit stride in the last dimension, q_stride = {batch,
 *             query, head} strides in elements
 *   indices   NULL: every token is attended.  Else device int32[batch]
 *             [queries][k], contiguous: only the listed positions, in any
 *             order, as ds_topk gives them for rows of index scores; entries
 *             that are negative or not below the query's limit are left out,
 *             a position listed twice counts twice
 *   out       device [batch][queries][heads][head_dim], contiguous
 *   lse       device float[batch][queries][heads], log of the sum of
 *             exp(scale * q k), or NULL
 *   workspace device, 16-byte aligned, of ds_kv4_attention_workspace bytes
 *             (NULL when that is 0)
 * A query that sees no token gives out = 0 and lse = -inf.  A probability times
 * a value scale is rounded to 11 significant bits (below 2^-28 of the largest of
 * each in its group of channels it is within 2^-39 of that), and q's channels
 * below 2^-25 of the row's largest are held to within 2^-35 of it; scores, maxima,
 * sums and outputs are held in 32 bits until they are rounded to `dtype`.  (A copy
 * into shared memory that does not end within a second, which no working GPU does,
 * is given up, and what depends on it is NaN.)
 */
int ds_kv4_attention(const ds_kv4_cache_t *cache, const int32_t *lengths, const int32_t *seqs,
                     int batch, int queries, int heads, int dtype, const void *q,
                     const int64_t *q_stride, const int32_t *indices, int k, float scale, void *out,
                     float *lse, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of ds_kv4_attention on the current device for these sizes, 0
 * where no sequence is shared by CTAs; k = 0 when every token is attended. */
int ds_kv4_attention_workspace(const ds_kv4_cache_t *cache, int batch, int queries, int heads,
                               int k, size_t *bytes);

/*
 * ds_kv4_chunk_attention -- the same for chunks of new tokens, as many for each
 * sequence as it has: prompts, or parts of them, read after what their sequences
 * hold already (a few tokens a sequence, one among them, are ds_kv4_attention's).
 *   starts    device int32[batch + 1]: rows [starts[b], starts[b + 1]) of q and out
 *             are the newest tokens of entry b's sequence, which ds_kv4_append has
 *             put into the cache; row j of n of a sequence of L tokens sees the
 *             tokens below max(0, L - n + 1 + j).  Below 0 they are read as 0,
 *             beyond `tokens` as that, and where they fall as the largest so far;
 *             rows of no entry are left as they were
 *   batch, seqs, lengths  as in ds_kv4_attention
 *   tokens    rows of q and out
 *   heads     query heads, a multiple of kv_heads
 *   dtype     of q and out: DS_BF16 or DS_FP16
 *   q         device, unit stride in the last dimension, q_stride = {token, head}
 *             strides in elements; 16 bytes at a time where these allow it
 *   scale     finite (from 2.35e38 on it is taken as that)
 *   out       device [tokens][heads][head_dim], contiguous, 16-byte aligned
 *   lse       device float[tokens][heads], or NULL
 *   workspace device, 16-byte aligned, of ds_kv4_chunk_attention_workspace bytes
 * max_pages * page_size is below 2^31 - 128.  A query that sees no token gives
 * out = 0 and lse = -inf.  Scores are sums in 32 bits of exact products, but for
 * channels beyond 16 bits: with DS_FP16, those of a token that has a key scale of 4096
 * or more are exact to 2^-18, and with DS_BF16 those of key scales from 64672 on to
 * 2^-13 of the channel.  A probability is rounded to 11
 * significant bits (below 2^-21 of the row's largest it is within 2^-32 of that), with
 * DS_FP16 to 22, and a value to 11 (below 2^-13 of the largest scale of its head, within 2^-24 of that);
 * maxima, sums and outputs are held in 32 bits.  A row with a NaN or an infinity
 * gives NaN if it sees a token.  (Waits are limited to a second, which no working
 * GPU takes; after that results are NaN.)
 */
int ds_kv4_chunk_attention(const ds_kv4_cache_t *cache, const int32_t *lengths, const int32_t *seqs,
                           const int32_t *starts, int batch, int64_t tokens, int heads, int dtype,
                           const void *q, const int64_t *q_stride, float scale, void *out, float *lse,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of ds_kv4_chunk_attention on the current device for these sizes. */
int ds_kv4_chunk_attention_workspace(const ds_kv4_cache_t *cache, int batch, int64_t tokens, int heads,
                                     size_t *bytes);

/* ---- pages -----------------------------------------------------------------
 * The page functions serve caches of any content: a page is page_bytes bytes
 * in each layer. */
typedef struct {
    void *pool;           /* layer l, page p at l * layer_stride + p * page_stride; 16-byte aligned */
    int64_t layer_stride; /* bytes, multiples of 16 */
    int64_t page_stride;
    int64_t page_bytes;   /* a multiple of 16 */
    int32_t layers;
    int32_t n_pages;
} ds_page_pool_t;

/* Who holds which page: refs[p] = sequences that hold page p (0: free).  Pages
 * and the entries of a list are 2^30 at most. */
typedef struct {
    int32_t *table;       /* [max_seqs][table_stride], -1 where a sequence has no page */
    int64_t table_stride;
    int32_t *lengths;     /* [max_seqs] tokens; a sequence holds ceil(length / page_size) pages */
    int32_t *refs;        /* [n_pages] */
    int32_t max_seqs;
    int32_t max_pages;
    int32_t page_size;
    int32_t n_pages;
} ds_page_book_t;

/* ds_pages_copy -- page dst[i] := page src[i], every layer, i < n (device
 * int32[n]).  Distinct destinations that are no sources; a pair with a page
 * out of range is skipped. */
int ds_pages_copy(const ds_page_pool_t *pool, const int32_t *src, const int32_t *dst, int n,
                  void *stream);

/* ds_pages_reserve -- sequence seqs[i] grows by tokens[i] tokens (device
 * int32[n]): its length is raised and it gets the pages it lacks, free pages
 * of lowest number first, in the list's order.  All or nothing:
 *   status  device int32[2] := {pages short, pages taken}; with pages short
 *           (too few free ones, or beyond max_pages of a row) nothing changes
 * Entries out of range, repeated sequences (after the first) and tokens < 1
 * are skipped.  The tokens' places are then written by ds_kv4_append. */
int ds_pages_reserve(const ds_page_book_t *book, const int32_t *seqs, const int32_t *tokens, int n,
                     int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/* ds_pages_fork -- sequence dst[i], empty before, becomes a copy of sequence
 * src[i]: it shares the full pages (their refs go up) and gets a copy of a
 * last page that is not full, so that no sequence writes into a shared page.
 * Free pages of lowest number first, in the list's order; several children of
 * one parent are fine.  All or nothing, and `status`, as in ds_pages_reserve.
 * Pairs out of range, with src = dst, with a dst that is not empty, or with a
 * dst that an earlier pair has, are skipped. */
int ds_pages_fork(const ds_page_pool_t *pool, const ds_page_book_t *book, const int32_t *src,
                  const int32_t *dst, int n, int32_t *status, void *workspace,
                  size_t workspace_bytes, void *stream);

/* ds_pages_free -- the sequences seqs[i] end: their pages' refs go down, their
 * table rows become -1 and their lengths 0.  Entries out of range and repeated
 * ones are skipped. */
int ds_pages_free(const ds_page_book_t *book, const int32_t *seqs, int n, void *stream);

/* ds_pages_compact -- the live pages (refs > 0) move to the front of the pool:
 * with N of them, the i-th free page below N takes the i-th live page at or
 * above N; table and refs follow (lengths is not used and may be NULL).
 *   remap   device int32[n_pages] := new number of each page, -1 of a free one
 *   status  device int32[2] := {N, pages moved} */
int ds_pages_compact(const ds_page_pool_t *pool, const ds_page_book_t *book, int32_t *remap,
                     int32_t *status, void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes that ds_pages_reserve and ds_pages_fork (n entries) and
 * ds_pages_compact (n = 0) need; 16-byte aligned. */
size_t ds_pages_workspace(int n_pages, int n);

#ifdef __cplusplus
}
#endif

#endif /* DS_KV4_H */
