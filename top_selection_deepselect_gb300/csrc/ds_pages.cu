// ds_pages.cu -- pages of a cache: copied, reserved, forked, freed and
// compacted.  Bookkeeping that numbers pages (which free page goes to whom) is
// done by one CTA in two sweeps over refs; the bytes are moved by the whole GPU
// in a second launch that reads what to move from the workspace.
#include "ds_kv4.h"

#include <cuda_runtime.h>
#include <limits.h>

#include "ds_device.cuh"
#include "ds_host.h"
#include "ds_topk.h"

namespace {

using ds::fail;
using ds::fail_cuda;

using Pool = ds_page_pool_t;
using Book = ds_page_book_t;

constexpr int kThreads = 1024;      // bookkeeping CTA
constexpr int kWarps = kThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kLoads = 4;  // 16-byte loads of a thread under way (2: 28.7 us for 500 pages, 4 and 8: 22.5)
constexpr int kChunk = kMoveThreads * 16 * kLoads;  // bytes a CTA moves at a time, at most

__device__ __forceinline__ int pages_of(const Book &b, int length)
{
    const long long room = (long long)b.max_pages * b.page_size;
    const long long n = length < 0 ? 0 : length > room ? room : length;
    return (int)((n + b.page_size - 1) / b.page_size);
}

// Sum over the CTA of `v`, and in *before the sum of the threads below.
template <typename T>
__device__ T block_scan(T v, T *before)
{
    __shared__ T sums[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    T x = v;
    for (int step = 1; step < 32; step *= 2) {
        const T y = __shfl_up_sync(~0u, x, step);
        if (lane >= step)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        sums[warp] = x;
    __syncthreads();
    T s = sums[lane];
    for (int step = 1; step < 32; step *= 2) {
        const T y = __shfl_up_sync(~0u, s, step);
        if (lane >= step)
            s += y;
    }
    const T below = __shfl_sync(~0u, s, (warp + 31) & 31);
    *before = x - v + (warp ? below : 0);
    return __shfl_sync(~0u, s, 31);
}

// The stretch of pages that a warp sweeps: [lo, hi).
__device__ __forceinline__ void stretch(int n_pages, int warp, int *lo, int *hi)
{
    const int each = ((n_pages + kWarps - 1) / kWarps + 31) / 32 * 32;
    const long long a = (long long)each * warp;
    *lo = a < n_pages ? (int)a : n_pages;
    *hi = a + each < n_pages ? (int)(a + each) : n_pages;
}

// Loads of a warp that are under way at once when it sweeps its stretch.
constexpr int kSweep = 8;

__device__ int count_live(const int32_t *refs, int lo, int hi)
{
    int n = 0;
#pragma unroll 8
    for (int p = lo + (threadIdx.x & 31); p < hi; p += 32)
        n += refs[p] > 0;
    for (int step = 16; step; step /= 2)
        n += __shfl_xor_sync(~0u, n, step);
    return n;
}

// Free pages in ascending order: the first `want` of them go to list[].
// Returns how many there are in all.
__device__ int list_free(const int32_t *refs, int n_pages, int want, int32_t *list)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int lo, hi, before;
    stretch(n_pages, warp, &lo, &hi);
    const int mine = hi - lo - count_live(refs, lo, hi);
    const int all = block_scan(lane == 0 ? mine : 0, &before);
    int at = __shfl_sync(~0u, before, 0);
    if (all >= want) {
        for (int p0 = lo; p0 < hi && at < want; p0 += 32 * kSweep) {
            int held[kSweep];
#pragma unroll
            for (int k = 0; k < kSweep; ++k) {
                const int p = p0 + 32 * k + lane;
                held[k] = p < hi ? refs[p] : 1;
            }
#pragma unroll
            for (int k = 0; k < kSweep; ++k) {
                const bool is_free = held[k] <= 0;
                const unsigned m = __ballot_sync(~0u, is_free);
                const int r = at + __popc(m & ((1u << lane) - 1));
                if (is_free && r < want)
                    list[r] = p0 + 32 * k + lane;
                at += __popc(m);
            }
        }
    }
    __syncthreads();
    return all;
}

// Places of an n-long list in the workspace.
struct Work {
    int32_t *pages;  // [n_pages]
    int32_t *a, *b;  // [n]
};

__device__ __forceinline__ Work work_of(int32_t *ws, int n_pages, int n)
{
    return {ws, ws + n_pages, ws + n_pages + n};
}

// A list entry's claim on a sequence: of equal entries the first keeps it.
// The sequence's length stands for the claim meanwhile, below any length.
__device__ __forceinline__ int claim(int i) { return INT32_MIN + i; }

__global__ void __launch_bounds__(kThreads)
reserve_kernel(Book book, const int32_t *seqs, const int32_t *tokens, int n, int32_t *status,
               int32_t *ws)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    const Work w = work_of(ws, book.n_pages, n);
    // lengths before the call, then the claims
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int s = seqs[i];
        w.a[i] = -1;
        if ((unsigned)s < (unsigned)book.max_seqs && tokens[i] > 0) {
            const int len = book.lengths[s];
            w.a[i] = max(len, 0);
            if (len < 0)
                book.lengths[s] = 0;    // below it a claim might not be seen
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (w.a[i] >= 0)
            atomicMin(book.lengths + seqs[i], claim(i));
    __syncthreads();
    // pages that each entry lacks; w.b becomes the first of its places in the
    // list (64-bit sums: the list may ask for far more than there is)
    long long total = 0, beyond = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        long long need = 0, before;
        if (i < n && w.a[i] >= 0) {
            if (book.lengths[seqs[i]] == claim(i)) {
                const long long len = (long long)w.a[i] + tokens[i];
                const long long want = (len + book.page_size - 1) / book.page_size;
                const int have = pages_of(book, w.a[i]);
                need = (want < book.max_pages ? want : book.max_pages) - have;
                beyond += want > book.max_pages ? want - book.max_pages : 0;
            } else {
                w.a[i] = -1;
            }
        }
        const long long sum = block_scan(need, &before);
        if (i < n)
            w.b[i] = (int)min(total + before, (long long)INT32_MAX);
        total += sum;
    }
    long long below;
    beyond = block_scan(beyond, &below);
    const int want = (int)min(total, (long long)INT32_MAX);
    const int available = list_free(book.refs, book.n_pages, want, w.pages);
    const long long lack = beyond + (total > available ? total - available : 0);
    const int missing = (int)min(lack, (long long)INT32_MAX);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        if (w.a[i] < 0)
            continue;
        const int s = seqs[i], old = w.a[i];
        if (missing) {
            book.lengths[s] = old;
            continue;
        }
        const int have = pages_of(book, old), end = pages_of(book, old + tokens[i]);
        for (int j = have; j < end; ++j) {
            const int page = w.pages[w.b[i] + j - have];
            book.table[s * book.table_stride + j] = page;
            book.refs[page] = 1;
        }
        book.lengths[s] = old + tokens[i];
    }
    if (threadIdx.x == 0) {
        status[0] = missing;
        status[1] = missing ? 0 : want;
    }
}

// First launch of a fork: which pairs count (w.a: the parent's length, -1 of a
// skipped pair) and which page each child's last tokens go to (w.b, -1 where
// the last page is full).
__global__ void __launch_bounds__(kThreads)
fork_plan_kernel(Book book, const int32_t *src, const int32_t *dst, int n, int32_t *status,
                 int32_t *ws)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    const Work w = work_of(ws, book.n_pages, n);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        const int s = src[i], d = dst[i];
        const bool ok = (unsigned)s < (unsigned)book.max_seqs &&
                        (unsigned)d < (unsigned)book.max_seqs && s != d && book.lengths[d] == 0;
        const long long room = (long long)book.max_pages * book.page_size;
        const int len = ok ? book.lengths[s] : 0;
        w.a[i] = !ok ? -1 : len < 0 ? 0 : len > room ? (int)room : len;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads)
        if (w.a[i] >= 0)
            atomicMin(book.lengths + dst[i], claim(i));
    __syncthreads();
    int total = 0;
    for (int i0 = 0; i0 < n; i0 += kThreads) {
        const int i = i0 + threadIdx.x;
        int need = 0;
        if (i < n && w.a[i] >= 0) {
            if (book.lengths[dst[i]] == claim(i))
                need = w.a[i] % book.page_size != 0;
            else
                w.a[i] = -1;
        }
        int before;
        const int sum = block_scan(need, &before);
        if (i < n)
            w.b[i] = need ? total + before : -1;
        total += sum;
    }
    const int available = list_free(book.refs, book.n_pages, total, w.pages);
    const int missing = max(total - available, 0);
    for (int i = threadIdx.x; i < n; i += kThreads) {
        if (w.a[i] < 0)
            continue;
        book.lengths[dst[i]] = missing ? 0 : w.a[i];
        if (missing)
            w.a[i] = -1;
        else if (w.b[i] >= 0)
            book.refs[w.b[i] = w.pages[w.b[i]]] = 1;
    }
    if (threadIdx.x == 0) {
        status[0] = missing;
        status[1] = missing ? 0 : total;
    }
}

// Bytes [at, at + size) of a page, size at most kChunk, by one CTA.
__device__ __forceinline__ void move_chunk(const Pool &pool, int layer, int from, int to, long long at,
                                           int size)
{
    const char *s = (const char *)pool.pool + layer * pool.layer_stride + from * pool.page_stride + at;
    char *d = (char *)pool.pool + layer * pool.layer_stride + to * pool.page_stride + at;
    uint4 v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int off = (j * kMoveThreads + threadIdx.x) * 16;
        if (off < size)
            v[j] = *reinterpret_cast<const uint4 *>(s + off);
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int off = (j * kMoveThreads + threadIdx.x) * 16;
        if (off < size)
            *reinterpret_cast<uint4 *>(d + off) = v[j];
    }
}

// How a page is cut: as few chunks as possible, of one size (the last one may
// be a little smaller).
struct Cut {
    long long chunks;
    int size;
    __host__ __device__ explicit Cut(long long page_bytes)
    {
        chunks = (page_bytes + kChunk - 1) / kChunk;
        size = (int)((page_bytes + chunks - 1) / chunks + 15) / 16 * 16;
    }
};

// All chunks of `moves` pages, every layer, spread over the grid.
template <typename From, typename To>
__device__ void move_pages(const Pool &pool, long long moves, From from, To to)
{
    const Cut cut(pool.page_bytes);
    const long long each = pool.layers * cut.chunks, items = moves * each;
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const long long m = it / each, rest = it - m * each;
        const int layer = (int)(rest / cut.chunks);
        const long long at = (rest - layer * cut.chunks) * cut.size;
        const long long left = pool.page_bytes - at;
        const int f = from(m), t = to(m);
        if ((unsigned)f < (unsigned)pool.n_pages && (unsigned)t < (unsigned)pool.n_pages)
            move_chunk(pool, layer, f, t, at, left < cut.size ? (int)left : cut.size);
    }
}

__global__ void __launch_bounds__(kMoveThreads)
copy_kernel(Pool pool, const int32_t *src, const int32_t *dst, int n)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    move_pages(pool, n, [&](long long m) { return src[m]; }, [&](long long m) { return dst[m]; });
}

// Second launch of a fork: table rows, refs of shared pages, last pages.
__global__ void __launch_bounds__(kMoveThreads)
fork_kernel(Pool pool, Book book, const int32_t *src, const int32_t *dst, int n, int32_t *ws)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    const Work w = work_of(ws, book.n_pages, n);
    const int pieces = (book.max_pages + kMoveThreads - 1) / kMoveThreads;
    for (long long it = blockIdx.x; it < (long long)n * pieces; it += gridDim.x) {
        const int i = (int)(it / pieces);
        const int col = (int)(it - (long long)i * pieces) * kMoveThreads + threadIdx.x;
        if (w.a[i] < 0 || col >= book.max_pages)
            continue;
        const int full = w.a[i] / book.page_size;
        int page = -1;
        if (col < full) {
            page = book.table[src[i] * book.table_stride + col];
            if ((unsigned)page < (unsigned)book.n_pages)
                atomicAdd(book.refs + page, 1);
        } else if (col == full) {
            page = w.b[i];
        }
        book.table[dst[i] * book.table_stride + col] = page;
    }
    move_pages(
        pool, n,
        [&](long long m) {
            return w.a[m] >= 0 && w.b[m] >= 0
                       ? book.table[src[m] * book.table_stride + w.a[m] / book.page_size] : -1;
        },
        [&](long long m) { return w.a[m] >= 0 ? w.b[m] : -1; });
}

__global__ void __launch_bounds__(kMoveThreads)
free_kernel(Book book, const int32_t *seqs)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    __shared__ int length;
    const int s = seqs[blockIdx.x];
    if ((unsigned)s >= (unsigned)book.max_seqs)
        return;
    // of repeated entries one finds the length, the others 0
    if (threadIdx.x == 0)
        length = atomicExch(book.lengths + s, 0);
    __syncthreads();
    const int used = pages_of(book, length);
    for (int col = threadIdx.x; length > 0 && col < book.max_pages; col += kMoveThreads) {
        int32_t *e = book.table + s * book.table_stride + col;
        const int page = *e;
        if (col < used && (unsigned)page < (unsigned)book.n_pages)
            atomicSub(book.refs + page, 1);
        *e = -1;
    }
}

// First launch of a compaction: remap[], and the moves (w.a holes, w.b movers).
__global__ void __launch_bounds__(kThreads)
compact_plan_kernel(Book book, int32_t *remap, int32_t *status, int32_t *holes, int32_t *movers)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    __shared__ int live_below;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    int lo, hi, before;
    stretch(book.n_pages, warp, &lo, &hi);
    const int mine = count_live(book.refs, lo, hi);
    const int live = block_scan(lane == 0 ? mine : 0, &before);
    before = __shfl_sync(~0u, before, 0);
    // live pages below number `live`
    if (lo <= live && (live < hi || (warp == kWarps - 1 && live == hi))) {
        const int n = before + count_live(book.refs, lo, live);
        if (lane == 0)
            live_below = n;
    }
    __syncthreads();
    const int moves = live - live_below;
    for (int p0 = lo, at = before; p0 < hi; p0 += 32 * kSweep) {
        int held[kSweep];
#pragma unroll
        for (int k = 0; k < kSweep; ++k) {
            const int p = p0 + 32 * k + lane;
            held[k] = p < hi ? book.refs[p] : 0;
        }
#pragma unroll
        for (int k = 0; k < kSweep; ++k) {
            const int p = p0 + 32 * k + lane;
            const bool is_live = held[k] > 0;
            const unsigned m = __ballot_sync(~0u, is_live);
            const int r = at + __popc(m & ((1u << lane) - 1));  // live pages below p
            at += __popc(m);
            if (is_live && p >= live)
                movers[r - live_below] = p;
            else if (p < hi)
                remap[p] = is_live ? p : -1;
            if (!is_live && p < hi && p < live)
                holes[p - r] = p;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < moves; i += kThreads)
        remap[movers[i]] = holes[i];
    if (threadIdx.x == 0) {
        status[0] = live;
        status[1] = moves;
    }
}

// Second launch of a compaction: bytes, table and refs.
__global__ void __launch_bounds__(kMoveThreads)
compact_kernel(Pool pool, Book book, const int32_t *remap, const int32_t *status,
               const int32_t *holes, const int32_t *movers)
{
    ds::dependent_grid_wait();
    ds::allow_dependent_grid();
    const int moves = status[1];
    const long long threads = (long long)gridDim.x * kMoveThreads;
    const long long me = (long long)blockIdx.x * kMoveThreads + threadIdx.x;
    for (long long i = me; i < moves; i += threads) {
        book.refs[holes[i]] = book.refs[movers[i]];
        book.refs[movers[i]] = 0;
    }
    const long long entries = (long long)book.max_seqs * book.max_pages;
    for (long long i = me; i < entries; i += threads) {
        const long long s = i / book.max_pages;
        int32_t *e = book.table + s * book.table_stride + (i - s * book.max_pages);
        const int page = *e;
        if ((unsigned)page < (unsigned)book.n_pages && remap[page] != page)
            *e = remap[page];
    }
    move_pages(pool, moves, [&](long long m) { return movers[m]; },
               [&](long long m) { return holes[m]; });
}

// ---- host ---------------------------------------------------------------------
// Most pages and list entries, so that sweeps that step past the end, by up to
// kThreads or 32 kSweep, stay in 32 bits.
constexpr int kMost = 1 << 30;

int check_pool(const Pool *p)
{
    if (!p)
        return fail(DS_EINVAL, "pool is NULL");
    if (p->layers < 1 || p->n_pages < 1 || p->page_bytes < 16 || p->page_bytes % 16 != 0)
        return fail(DS_EINVAL,
                    "layers = %d and n_pages = %d must be >= 1 and page_bytes = %lld a positive "
                    "multiple of 16",
                    p->layers, p->n_pages, (long long)p->page_bytes);
    if (p->page_bytes > 1LL << 40)
        return fail(DS_EUNSUPPORTED, "page_bytes = %lld is above 2^40", (long long)p->page_bytes);
    if (p->page_stride % 16 != 0 || p->page_stride < p->page_bytes || p->layer_stride % 16 != 0)
        return fail(DS_EINVAL,
                    "page_stride = %lld must be a multiple of 16 of at least page_bytes = %lld, and "
                    "layer_stride = %lld a multiple of 16",
                    (long long)p->page_stride, (long long)p->page_bytes, (long long)p->layer_stride);
    if (!p->pool || (uintptr_t)p->pool % 16 != 0)
        return fail(DS_EINVAL, "the pool must be non-NULL and 16-byte aligned");
    return DS_OK;
}

int check_book(const Book *b, bool lengths)
{
    if (!b)
        return fail(DS_EINVAL, "book is NULL");
    if (b->max_seqs < 1 || b->max_pages < 1 || b->n_pages < 1 || b->page_size < 1)
        return fail(DS_EINVAL,
                    "max_seqs = %d, max_pages = %d, n_pages = %d and page_size = %d must all be >= 1",
                    b->max_seqs, b->max_pages, b->n_pages, b->page_size);
    if (b->n_pages > kMost)
        return fail(DS_EUNSUPPORTED, "n_pages = %d is above 2^30", b->n_pages);
    if ((long long)b->max_pages * b->page_size >= 1LL << 31)
        return fail(DS_EINVAL, "max_pages * page_size = %lld is not below 2^31",
                    (long long)b->max_pages * b->page_size);
    if (b->table_stride < b->max_pages)
        return fail(DS_EINVAL, "table_stride = %lld is below max_pages = %d",
                    (long long)b->table_stride, b->max_pages);
    if (!b->table || !b->refs || (lengths && !b->lengths))
        return fail(DS_EINVAL, "table, lengths and refs must be non-NULL");
    return DS_OK;
}

int check_both(const Pool *p, const Book *b)
{
    if (p->n_pages != b->n_pages)
        return fail(DS_EINVAL, "the pool has %d pages, the book %d", p->n_pages, b->n_pages);
    return DS_OK;
}

int check_list(int n, bool given)
{
    if (n < 0)
        return fail(DS_EINVAL, "n = %d is negative", n);
    if (n > kMost)
        return fail(DS_EUNSUPPORTED, "n = %d is above 2^30", n);
    if (n > 0 && !given)
        return fail(DS_EINVAL, "the lists must be non-NULL when n > 0");
    return DS_OK;
}

int check_work(const void *ws, size_t bytes, size_t need)
{
    if (!ws || (uintptr_t)ws % 16 != 0 || bytes < need)
        return fail(DS_EINVAL, "workspace must be 16-byte aligned and hold %zu bytes (%zu given)",
                    need, bytes);
    return DS_OK;
}

// CTAs that move pages: no more than there are chunks, and many more than fit at
// once, so that SMs nearer to their memory take more of them (500 pages of 37 KB
// in four layers: 22.5 us with 8, 64 and 1024 a SM; a compaction of 8192, whose
// moves the host only knows a bound of: 175, 169 and 216).
int move_grid(long long items, unsigned *grid)
{
    int dev = 0, sms = 0;
    const int rc = ds::current_device(&dev, &sms);
    if (rc != DS_OK)
        return rc;
    const long long most = 64LL * sms;
    *grid = (unsigned)(items < 1 ? 1 : items < most ? items : most);
    return DS_OK;
}

long long chunks_of(const Pool &p) { return p.layers * Cut(p.page_bytes).chunks; }

int finish(const char *what, cudaError_t e)
{
    return e == cudaSuccess ? DS_OK : fail_cuda(e, what);
}

}  // namespace

extern "C" {

size_t ds_pages_workspace(int n_pages, int n)
{
    const size_t p = n_pages > 0 ? (size_t)n_pages : 0, q = n > 0 ? (size_t)n : 0;
    return (2 * p + 2 * q + 4) * sizeof(int32_t);
}

int ds_pages_copy(const ds_page_pool_t *pool, const int32_t *src, const int32_t *dst, int n,
                  void *stream)
{
    ds::g_detail[0] = '\0';
    int rc = check_pool(pool);
    if (rc == DS_OK)
        rc = check_list(n, src && dst);
    unsigned grid = 0;
    if (rc != DS_OK || n == 0)
        return rc;
    if ((rc = move_grid(n * chunks_of(*pool), &grid)) != DS_OK)
        return rc;
    return finish("ds_pages_copy", ds::launch_overlapped(copy_kernel, grid, kMoveThreads, 0,
                                                         (cudaStream_t)stream, *pool, src, dst, n));
}

int ds_pages_reserve(const ds_page_book_t *book, const int32_t *seqs, const int32_t *tokens, int n,
                     int32_t *status, void *workspace, size_t workspace_bytes, void *stream)
{
    ds::g_detail[0] = '\0';
    int rc = check_book(book, true);
    if (rc == DS_OK)
        rc = check_list(n, seqs && tokens);
    if (rc == DS_OK && !status)
        rc = fail(DS_EINVAL, "status must be non-NULL");
    if (rc == DS_OK)
        rc = check_work(workspace, workspace_bytes, ds_pages_workspace(book->n_pages, n));
    if (rc != DS_OK)
        return rc;
    return finish("ds_pages_reserve",
                  ds::launch_overlapped(reserve_kernel, 1, kThreads, 0, (cudaStream_t)stream, *book, seqs,
                                        tokens, n, status, (int32_t *)workspace));
}

int ds_pages_fork(const ds_page_pool_t *pool, const ds_page_book_t *book, const int32_t *src,
                  const int32_t *dst, int n, int32_t *status, void *workspace,
                  size_t workspace_bytes, void *stream)
{
    ds::g_detail[0] = '\0';
    int rc = check_pool(pool);
    if (rc == DS_OK)
        rc = check_book(book, true);
    if (rc == DS_OK)
        rc = check_both(pool, book);
    if (rc == DS_OK)
        rc = check_list(n, src && dst);
    if (rc == DS_OK && !status)
        rc = fail(DS_EINVAL, "status must be non-NULL");
    if (rc == DS_OK)
        rc = check_work(workspace, workspace_bytes, ds_pages_workspace(book->n_pages, n));
    unsigned grid = 0;
    if (rc == DS_OK)
        rc = move_grid(n * chunks_of(*pool), &grid);
    if (rc != DS_OK)
        return rc;
    int32_t *ws = (int32_t *)workspace;
    cudaError_t e = ds::launch_overlapped(fork_plan_kernel, 1, kThreads, 0, (cudaStream_t)stream, *book,
                                          src, dst, n, status, ws);
    if (e == cudaSuccess && n > 0)
        e = ds::launch_overlapped(fork_kernel, grid, kMoveThreads, 0, (cudaStream_t)stream, *pool, *book,
                                  src, dst, n, ws);
    return finish("ds_pages_fork", e);
}

int ds_pages_free(const ds_page_book_t *book, const int32_t *seqs, int n, void *stream)
{
    ds::g_detail[0] = '\0';
    int rc = check_book(book, true);
    if (rc == DS_OK)
        rc = check_list(n, seqs != nullptr);
    if (rc != DS_OK || n == 0)
        return rc;
    return finish("ds_pages_free", ds::launch_overlapped(free_kernel, (unsigned)n, kMoveThreads, 0,
                                                         (cudaStream_t)stream, *book, seqs));
}

int ds_pages_compact(const ds_page_pool_t *pool, const ds_page_book_t *book, int32_t *remap,
                     int32_t *status, void *workspace, size_t workspace_bytes, void *stream)
{
    ds::g_detail[0] = '\0';
    int rc = check_pool(pool);
    if (rc == DS_OK)
        rc = check_book(book, false);
    if (rc == DS_OK)
        rc = check_both(pool, book);
    if (rc == DS_OK && (!remap || !status))
        rc = fail(DS_EINVAL, "remap and status must be non-NULL");
    if (rc == DS_OK)
        rc = check_work(workspace, workspace_bytes, ds_pages_workspace(book->n_pages, 0));
    unsigned grid = 0;
    if (rc == DS_OK)
        rc = move_grid(pool->n_pages / 2 * chunks_of(*pool), &grid);
    if (rc != DS_OK)
        return rc;
    int32_t *holes = (int32_t *)workspace, *movers = holes + book->n_pages;
    cudaError_t e = ds::launch_overlapped(compact_plan_kernel, 1, kThreads, 0, (cudaStream_t)stream,
                                          *book, remap, status, holes, movers);
    if (e == cudaSuccess)
        e = ds::launch_overlapped(compact_kernel, grid, kMoveThreads, 0, (cudaStream_t)stream, *pool,
                                  *book, remap, status, holes, movers);
    return finish("ds_pages_compact", e);
}

}  // extern "C"
