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

// Lays the call out: what every entry holds, blocks of rows with their places on
// the line, and which block each CTA begins in.  A thread an entry looks it up, a
// warp an entry works on its blocks.  kPlanThreads entries
// at a time, in shared memory; where there are more they are looked up twice.
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const __grid_constant__ Args p)
{
    __shared__ long long scratch[kPlanThreads / 32];
    __shared__ int scratch_int[kPlanThreads / 32];
    __shared__ Entry entries[kPlanThreads];
    __shared__ long long places[kPlanThreads];      // of an entry
    __shared__ int counts[kPlanThreads];            // blocks of an entry
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = kPlanThreads / 32;
    dependent_grid_wait();
    allow_dependent_grid();

    // Entries b0 on: looked up, with starts as far as they rise, so that no two share a
    // row; `most` is the largest start before.  Then their blocks and places.
    auto look = [&](int b0, int most) -> int {
        const int b = b0 + threadIdx.x;
        const bool in = b < p.a.batch;
        auto larger = [](int x, int y) { return x > y ? x : y; };
        const int first = in ? start_of(p, b) : 0, next = in ? start_of(p, b + 1) : 0;
        Entry e = {};
        if (in)
            e = entry_of(p, b);
        int before;
        const int all = scan_all(first, 0, larger, &before, scratch_int);
        e.start = larger(most, larger(before, first));
        const int end = larger(e.start, next);
        e.n = in ? end - e.start : 0;
        entries[threadIdx.x] = e;
        __syncthreads();
        for (int i = warp; i < kPlanThreads && b0 + i < p.a.batch; i += warps) {
            Block k = {};
            k.n = entries[i].n;
            k.len = entries[i].len;
            const int rows = k.n * p.group, blocks = (int)(((long long)rows + p.rows - 1) / p.rows);
            long long cost = 0;
            for (int j = lane; j < blocks; j += 32) {
                k.row0 = j * p.rows;
                cost += cost_of(span_of(k, p.by_group, p.group, p.rows));
            }
#pragma unroll
            for (int step = 16; step; step /= 2)
                cost += __shfl_xor_sync(~0u, cost, step);
            if (lane == 0) {
                counts[i] = blocks;
                places[i] = cost;
            }
        }
        __syncthreads();
        return larger(most, all);
    };
    // Exclusive sums over these entries' places and blocks, and their totals.
    auto add_up = [&](int b0, long long *place, int *block) {
        auto plus = [](auto x, auto y) { return x + y; };
        const bool in = b0 + (int)threadIdx.x < p.a.batch;
        long long place_before;
        int block_before;
        const long long place_all = scan_all(in ? places[threadIdx.x] : 0LL, 0LL, plus, &place_before, scratch);
        const int block_all = scan_all(in ? counts[threadIdx.x] : 0, 0, plus, &block_before, scratch_int);
        __syncthreads();
        places[threadIdx.x] = *place + place_before;
        counts[threadIdx.x] = *block + block_before;
        __syncthreads();
        *place += place_all;
        *block += block_all;
    };
    auto write = [&](int b0, long long per) {
        for (int e = warp; e < kPlanThreads && b0 + e < p.a.batch; e += warps) {
            Block k = {};
            k.seq = entries[e].seq;
            k.start = entries[e].start;
            k.n = entries[e].n;
            k.len = entries[e].len;
            const int rows = k.n * p.group, count = (int)(((long long)rows + p.rows - 1) / p.rows);
            long long place = places[e];
            const int number = counts[e];
            for (int i0 = 0; i0 < count; i0 += 32) {
                const int i = i0 + lane;
                k.row0 = i * p.rows;
                const int cost = i < count ? cost_of(span_of(k, p.by_group, p.group, p.rows)) : 0;
                long long upto = cost;
#pragma unroll
                for (int step = 1; step < 32; step *= 2) {
                    const long long y = __shfl_up_sync(~0u, upto, step);
                    if (lane >= step)
                        upto += y;
                }
                if (i < count) {
                    k.place = place + upto - cost;
                    p.blocks[number + i] = k;
                    const long long from = k.place * p.c.kv_heads, to = from + (long long)cost * p.c.kv_heads;
                    for (long long c = (from + per - 1) / per; c * per < to; ++c)
                        p.first[c] = number + i;
                }
                place += __shfl_sync(~0u, upto, 31);
            }
        }
        __syncthreads();
    };

    long long place = 0;
    int block = 0, most = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += kPlanThreads) {
        most = look(b0, most);
        add_up(b0, &place, &block);
    }
    Head h;
    h.all = place * p.c.kv_heads;
    h.per = places_of_cta(p, h.all);
    h.blocks = block;
    h.pad = 0;
    if (threadIdx.x == 0)
        *p.head = h;
    if (p.a.batch <= kPlanThreads) {          // all of it is still here
        write(0, h.per);
        return;
    }
    place = 0;
    block = most = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += kPlanThreads) {
        most = look(b0, most);
        add_up(b0, &place, &block);
        write(b0, h.per);
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
    const double units = (double)blocks * p.c.kv_heads;
    p.few = p.a.batch <= kFew && blocks <= kFew && units * (room / 64 + 1) <= 16.0 * sms;
    p.whole = room <= 512;                 // eight tiles
    const double most = p.whole ? units : units * (kUnitCost + 8 * (room / 64 + 1)) / kLeast + 1;
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
    p.blocks = (Block *)take(blocks * sizeof(Block));
    p.partial = (float *)take(p.whole ? 0 : 2ULL * p.ctas * p.rows * (head_dim + 2) * sizeof(float));
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
    if (!p.few) {
        const cudaError_t e = launch_overlapped(chunk::plan_kernel, 1, chunk::kPlanThreads, 0, stream, p);
        if (e != cudaSuccess)
            return e;
    }
    return head_dim == 64    ? launch_chunk_64(p, dev, p.ctas, stream)
           : head_dim == 128 ? launch_chunk_128(p, dev, p.ctas, stream)
                             : launch_chunk_256(p, dev, p.ctas, stream);
}

}  // namespace kv4
}  // namespace ds
