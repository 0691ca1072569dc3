// ds_kv4_chunk.cu -- attention of chunks: the planning launch, the workspace, and
// the choice of the head dimension's instantiation.
#include "ds_kv4_chunk.h"

#include "ds_device.cuh"
#include "ds_host.h"

namespace ds {
namespace kv4 {

cudaError_t launch_chunk_64(const chunk::Args &p, int dev, int ctas, cudaStream_t stream);
cudaError_t launch_chunk_128(const chunk::Args &p, int dev, int ctas, cudaStream_t stream);
cudaError_t launch_chunk_256(const chunk::Args &p, int dev, int ctas, cudaStream_t stream);

namespace chunk {
namespace {

constexpr int kPlanThreads = 1024;
// Places of a CTA where units are cut: not more parts to join than the work is worth.
constexpr int kLeast = 96;

// Of a value a thread: what `combine` makes of all threads', and in *before of those below.
template <typename V, typename F>
__device__ V scan_all(V v, V none, F combine, V *before, V *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    V x = v;
#pragma unroll
    for (int step = 1; step < 32; step *= 2) {
        const V y = __shfl_up_sync(~0u, x, step);
        if (lane >= step)
            x = combine(y, x);
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = x;
    __syncthreads();
    V below = none, all = none;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp)
            below = combine(below, scratch[w]);
        all = combine(all, scratch[w]);
    }
    const V left = __shfl_up_sync(~0u, x, 1);
    *before = lane == 0 ? below : combine(below, left);
    return all;
}

// The block of rows that begins at row0 of entry b.
__device__ __forceinline__ Block block_of(const Args &p, int b, int row0)
{
    Block k;
    k.place = 0;
    k.seq = p.a.seqs ? p.a.seqs[b] : b;
    k.start = p.starts[b];
    k.n = p.starts[b + 1] - k.start;
    k.len = 0;
    if ((unsigned)k.seq < (unsigned)p.c.max_seqs) {
        const int n = p.a.lengths[k.seq];
        const long long room = (long long)p.c.max_pages * p.c.page_size;
        k.len = n < 0 ? 0 : n > room ? (int)room : n;
    }
    k.row0 = row0;
    k.pad = 0;
    return k;
}

// Lays the call out: what every entry holds, blocks of rows with their places on
// the line, and which block each CTA begins in.  A warp an entry.
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ Args p)
{
    __shared__ long long scratch[kPlanThreads / 32];
    __shared__ int scratch_int[kPlanThreads / 32];
    __shared__ long long per_shared;
    dependent_grid_wait();
    allow_dependent_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = kPlanThreads / 32;

    // starts as far as they rise, so that no two entries share a row
    int most = 0;
    for (int i0 = 0; i0 <= p.a.batch; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        const int given = i <= p.a.batch ? p.a.starts[i] : 0;
        const int mine = given < 0 ? 0 : given > p.a.tokens ? p.a.tokens : given;
        int before;
        auto larger = [](int a, int b) { return a > b ? a : b; };
        const int all = scan_all(mine, 0, larger, &before, scratch_int);
        if (i <= p.a.batch)
            p.starts[i] = larger(most, larger(before, mine));
        most = larger(most, all);
    }
    __syncthreads();

    for (int b = warp; b < p.a.batch; b += warps) {
        const Block k = block_of(p, b, 0);
        const int rows = k.n * p.group, blocks = rows / p.rows + (rows % p.rows != 0);
        long long cost = 0;
        for (int i = lane; i < blocks; i += 32) {
            Block x = k;
            x.row0 = i * p.rows;
            cost += cost_of(span_of(x, p.group, p.rows));
        }
#pragma unroll
        for (int step = 16; step; step /= 2)
            cost += __shfl_xor_sync(~0u, cost, step);
        if (lane == 0) {
            p.counts[b] = blocks;
            p.places[b] = cost;
        }
    }
    __syncthreads();

    long long places = 0;
    int blocks = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        auto sum = [](auto x, auto y) { return x + y; };
        long long place_before;
        int block_before;
        const long long place_all =
            scan_all(b < p.a.batch ? p.places[b] : 0LL, 0LL, sum, &place_before, scratch);
        const int block_all = scan_all(b < p.a.batch ? p.counts[b] : 0, 0, sum, &block_before, scratch_int);
        if (b < p.a.batch) {
            p.places[b] = places + place_before;
            p.counts[b] = blocks + block_before;
        }
        places += place_all;
        blocks += block_all;
    }
    if (threadIdx.x == 0) {
        Head h;
        h.all = places * p.c.kv_heads;
        h.per = (h.all + p.ctas - 1) / p.ctas;
        h.per = h.per > kLeast ? h.per : kLeast;
        h.blocks = blocks;
        h.pad = 0;
        *p.head = h;
        per_shared = h.per;
    }
    __syncthreads();

    const long long per = per_shared;
    for (int b = warp; b < p.a.batch; b += warps) {
        const Block k = block_of(p, b, 0);
        const int rows = k.n * p.group, count = rows / p.rows + (rows % p.rows != 0);
        long long place = p.places[b];
        const int number = p.counts[b];
        for (int i0 = 0; i0 < count; i0 += 32) {
            const int i = i0 + lane;
            Block x = k;
            x.row0 = i * p.rows;
            const int cost = i < count ? cost_of(span_of(x, p.group, p.rows)) : 0;
            long long upto = cost;
#pragma unroll
            for (int step = 1; step < 32; step *= 2) {
                const long long y = __shfl_up_sync(~0u, upto, step);
                if (lane >= step)
                    upto += y;
            }
            if (i < count) {
                x.place = place + upto - cost;
                p.blocks[number + i] = x;
                const long long from = x.place * p.c.kv_heads, to = from + (long long)cost * p.c.kv_heads;
                for (long long c = (from + per - 1) / per; c * per < to; ++c)
                    p.first[c] = number + i;
            }
            place += __shfl_sync(~0u, upto, 31);
        }
    }
}

size_t rounded(size_t n) { return (n + 255) / 256 * 256; }

// Sizes that follow from the call, and the workspace's parts.
size_t lay_out(Args &p, int head_dim, int sms, unsigned char *base)
{
    p.group = p.a.heads / p.c.kv_heads;
    p.rows = tiles_of_rows(head_dim) * 128;
    const long long blocks = (long long)p.a.tokens * p.group / p.rows + p.a.batch;
    // no more CTAs than the largest possible line has work for
    const double room = (double)p.c.max_pages * p.c.page_size;
    const double most = (double)blocks * p.c.kv_heads * (kUnitCost + 8 * (room / 64 + 1)) / kLeast + 1;
    p.ctas = most < sms ? (int)most : sms;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        unsigned char *here = base + at;
        at += rounded(bytes);
        return here;
    };
    p.head = (Head *)take(sizeof(Head));
    p.splits = (Split *)take(p.ctas * sizeof(Split));
    p.first = (int *)take(p.ctas * sizeof(int));
    p.starts = (int *)take((p.a.batch + 1LL) * sizeof(int));
    p.places = (long long *)take(p.a.batch * sizeof(long long));
    p.counts = (int *)take(p.a.batch * sizeof(int));
    p.blocks = (Block *)take(blocks * sizeof(Block));
    p.partial = (float *)take(2ULL * p.ctas * p.rows * (head_dim + 2) * sizeof(float));
    return at;
}

}  // namespace
}  // namespace chunk

size_t chunk_workspace(const Cache &c, int head_dim, const Chunk &a, int sms)
{
    chunk::Args p = {};
    p.c = c;
    p.a = a;
    return chunk::lay_out(p, head_dim, sms, nullptr);
}

cudaError_t launch_chunk(const Cache &c, int head_dim, const Chunk &a, void *workspace, int dev, int sms,
                         cudaStream_t stream)
{
    chunk::Args p = {};
    p.c = c;
    p.a = a;
    chunk::lay_out(p, head_dim, sms, (unsigned char *)workspace);
    p.by_group.set(p.group);
    p.run = 1;
    while (p.run < 8 && c.page_size % (2 * p.run) == 0)
        p.run *= 2;
    p.q_vector = ((uintptr_t)a.q | a.q_query * 2 | a.q_head * 2) % 16 == 0;
    const cudaError_t e = launch_overlapped(chunk::plan_kernel, 1, chunk::kPlanThreads, 0, stream, p);
    if (e != cudaSuccess)
        return e;
    return head_dim == 64    ? launch_chunk_64(p, dev, p.ctas, stream)
           : head_dim == 128 ? launch_chunk_128(p, dev, p.ctas, stream)
                             : launch_chunk_256(p, dev, p.ctas, stream);
}

}  // namespace kv4
}  // namespace ds
