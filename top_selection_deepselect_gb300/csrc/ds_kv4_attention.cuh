// ds_kv4_attention.cuh -- attention over the 4-bit cache on the tensor cores.
//
// Decoding reads each record once and does little with it: 4.5 bits a channel,
// 2 x D products for each query head.  The bound is HBM as long as turning
// codes into operands and the softmax cost few instructions, so everything
// here is laid out for that.
//
// Codes become operands with one logical operation and one packed addition.  A
// code u (0..15) in the low bits of an fp16 of value 1024 makes it 1024 + u, in
// bits 4..7 it makes it 1024 + 16 u; subtracting 1032 or 1152 leaves u - 8 or
// 16 (u - 8), exactly.  A word of eight codes gives four operand registers with
// one shift and four of each, no conversion.  The factor 16 is taken back by
// the query (2^-4 there) and the epilogue.  Without the addition, on the fp16
// subnormals u 2^-24 and with -8 sum(q) as the accumulator's start, scores were
// off by up to 2^-17 of the sum of their terms' sizes: the matrix unit aligns
// its addends by exponent and cuts them off below the largest one.
//
// Both products have tokens or channels as the 16 rows and up to 8 (query,
// head) rows of one key/value head as the 8 columns of m16n8k16:
//   S^T = K Q^T   rows are tokens; for each group of 32 channels the sum is
//                 multiplied by the token's key scale in 32 bits
//   O^T = V^T P^T rows are channels; the probabilities carry the value scale
//                 of (token, group): fp16(p * scale), the only rounding of the
//                 inner loop.  2^-11 relative on each token's share, less than
//                 the output's own rounding; 32-bit operands would halve the
//                 rate of the matrix instructions.  Denominators are summed in
//                 32 bits from unrounded p.
// The transposition of P between the two is one movmatrix per 8 x 8.  m64+ tile
// instructions (tcgen05) would leave 7/8 of their rows empty at 8 query rows and
// need the operands written back to shared memory after the expansion.
//
// Work is cut into tiles of kTile tokens; all tiles of all (sequence, head)
// units stand in one line that is divided evenly among the CTAs, whatever the
// lengths are; they are read on the device, so that the host needs to know
// nothing.  A CTA's warps take its tiles in turn, each with its own ring of
// asynchronous copies, running maximum, sum and output, and meet only at the
// end of a unit.  A unit cut between CTAs leaves partial results in the
// workspace; a second launch joins them in a fixed order.
#pragma once

#include <type_traits>

#include "ds_device.cuh"
#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {

constexpr int kAttendWarps = 8;
constexpr int kAttendThreads = kAttendWarps * 32;

// Quotient by a fixed divisor of numbers below 2^31.
struct Divider {
    unsigned mul;
    int shift;
    void set(int d)
    {
        int l = 0;
        while ((1LL << l) < d)
            ++l;
        mul = (unsigned)(((1ULL << (31 + l)) + d - 1) / d);
        shift = 31 + l;
    }
    __device__ __forceinline__ int operator()(int n) const
    {
        return (int)((unsigned long long)(unsigned)n * mul >> shift);
    }
};

// Shape of one instantiation.
template <int D, int NT>
struct Shape {
    static constexpr int kGroups = D / kGroup;
    static constexpr int kStretches = D > 128 ? D / 128 : 1;   // of up to 128 channels
    static constexpr int kPer = kGroups / kStretches;           // groups of a stretch
    static constexpr int kRows = 8 * NT;
    static constexpr int kMT = D == 256 ? 1 : 2;                // 16-token steps of a tile
    static constexpr int kTile = 16 * kMT;
    static constexpr int kRecord = record_bytes(D);
    // Distance of records in shared memory: the operand loads of a warp then
    // touch every bank once.
    static constexpr int kStride = D == 256 ? kRecord + 16 : kRecord;
    static constexpr int kStageBytes = kTile * kStride;
    static constexpr bool kTwoCtas = D * NT <= 256;             // output registers of a thread: D NT / 4
    static constexpr int kStages = D == 64 ? 4 : D == 128 ? (kTwoCtas ? 3 : 5) : (kTwoCtas ? 2 : 4);
    static constexpr int kOutStride = D + 4;                    // floats of an output row in shared memory
    // A warp's ring; at a unit's end its output, the rows' maxima and sums.
    static constexpr int kOffMax = kRows * kOutStride * 4;
    static constexpr int kOffSum = kOffMax + kRows * 4;
    static constexpr int kWarpBytes = kStages * kStageBytes > kOffSum + kRows * 4
                                          ? kStages * kStageBytes : kOffSum + kRows * 4;
    // shared memory behind the rings
    static constexpr int kOffQ = kAttendWarps * kWarpBytes;            // query operands
    static constexpr int kOffFactor = kOffQ + kGroups * 2 * NT * 32 * 8;
    static constexpr int kOffLimit = kOffFactor + kRows * 4;
    static constexpr int kOffBarrier = (kOffLimit + kRows * 4 + 15) / 16 * 16;
    static constexpr int kOffMask = kOffBarrier + kAttendWarps * kStages * 8;
    static constexpr int kOffScan = (kOffMask + kAttendWarps * kStages * 4 + 15) / 16 * 16;
    static constexpr int kSmem = (kOffScan + 16 * 8 + 15) / 16 * 16;
    static constexpr int kPartial = kRows * (D + 2);                   // floats of a partial result
};

struct AttendArgs {
    Cache c;
    Attend a;
    Divider by_page;
    long long sel_tiles;  // tiles of a unit when tokens are listed
    int run;              // tokens of a tile that lie side by side in a page, a power of two
    int group;            // query heads of a key/value head
    int rows;             // query rows of a unit before it is cut into blocks
    int blocks;           // blocks of kRows rows
    int units;            // units of a batch entry
};

__device__ __forceinline__ uint32_t shared_address(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}

// Arrival barriers of the rings: one arrival (lane 0's, with the bytes to
// come) and the bytes themselves complete a phase.
__device__ __forceinline__ void barrier_init(uint32_t bar)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void barrier_expect(uint32_t bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Whether the phase ended; gives up after kPatience tries (far beyond any
// copy's time), so that a copy that never ends cannot hang the GPU.
constexpr int kPatience = 1 << 20;
__device__ __forceinline__ bool barrier_wait(uint32_t bar, unsigned phase)
{
    for (int i = 0; i < kPatience; ++i) {
        unsigned done;
        asm volatile("{\n\t.reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done) : "r"(bar), "r"(phase) : "memory");
        if (done)
            return true;
    }
    return false;
}

// Asynchronous copy of `bytes` (a multiple of 16) from global to shared memory.
__device__ __forceinline__ void copy_bulk(uint32_t dst, const void *src, unsigned bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(bar) : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
                 "{%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// u - 8 of the codes in the low four bits of each half, and 16 (u - 8) of those
// in the four bits above.
__device__ __forceinline__ uint32_t low_codes(uint32_t w)
{
    uint32_t x, y;
    asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x) : "r"(w));  // (w & mask) | 1024
    asm("add.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xe408e408u));         // - 1032
    return y;
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w)
{
    uint32_t x, y;
    asm("lop3.b32 %0, %1, 0x00f000f0, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
    asm("add.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xe480e480u));         // - 1152
    return y;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi)
{
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], const unsigned char *p)
{
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
    } else {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
}

// Scales of G groups as floats.
template <int G>
__device__ __forceinline__ void load_scales(float (&s)[G], const unsigned char *p)
{
    uint32_t w[G / 2];
    load_words(w, p);
#pragma unroll
    for (int i = 0; i < G / 2; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        s[2 * i] = f.x, s[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ int sequence_of(const AttendArgs &p, int b)
{
    return p.a.seqs ? __ldg(p.a.seqs + b) : b;
}

__device__ __forceinline__ int length_of(const AttendArgs &p, int seq)
{
    if ((unsigned)seq >= (unsigned)p.c.max_seqs)
        return 0;
    const int n = __ldg(p.a.lengths + seq);
    const long long room = (long long)p.c.max_pages * p.c.page_size;
    return n < 0 ? 0 : n > room ? (int)room : n;
}

// Tiles of every unit of batch entry b: at least one, so that rows that see
// nothing are written too.
template <int kTile, bool kListed>
__device__ __forceinline__ long long tiles_of(const AttendArgs &p, int b)
{
    if (kListed)
        return p.sel_tiles;
    const int n = length_of(p, sequence_of(p, b));
    return n > kTile ? (n + kTile - 1LL) / kTile : 1;
}

// Sum over the CTA (a power of two of at most 8 warps), and in *before the sum
// of the threads below.
__device__ __forceinline__ long long scan_cta(long long v, long long *before, long long *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = blockDim.x / 32;
    long long x = v;
#pragma unroll
    for (int step = 1; step < 32; step *= 2) {
        const long long y = __shfl_up_sync(~0u, x, step);
        if (lane >= step)
            x += y;
    }
    __syncthreads();
    if (lane == 31)
        scratch[warp] = x;
    __syncthreads();
    long long below = 0, all = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp)
            below += scratch[w];
        all += scratch[w];
    }
    *before = below + x - v;
    return all;
}

// The line of work: each unit takes kUnitCost places and one for each of its
// tiles.  A unit's start and end (its queries, the first copies' latency, the
// meeting of the warps) cost a CTA as much as some tiles do; without these
// places the CTA that met 24 empty sequences in a row took four times as long
// as the others.
constexpr int kUnitCost = 12;

// Places of the line for each of `ctas` CTAs: two tiles a warp at least, so
// that there are not more parts to join than the work is worth.
__device__ __forceinline__ long long places_per_cta(long long all, int ctas)
{
    const long long even = (all + ctas - 1) / ctas;
    return even > 2 * kAttendWarps ? even : 2 * kAttendWarps;
}

// The line's length and, for batch entry `entry`, its first place; with entry
// < 0 the entry that place `per * cta` belongs to and that one's first place.
struct Line {
    long long all, per, first;
    int entry;
};

template <int kTile, bool kListed>
__device__ __forceinline__ Line line_of(const AttendArgs &p, int ctas, int cta, int entry,
                                        long long *scratch)
{
    Line n;
    if (kListed) {
        const long long each = (p.sel_tiles + kUnitCost) * p.units;
        n.all = each * p.a.batch;
        n.per = places_per_cta(n.all, ctas);
        n.entry = entry >= 0 ? entry : (int)(n.per * cta / each);
        n.first = n.entry * each;
        return n;
    }
    const bool once = p.a.batch <= (int)blockDim.x;   // then one scan answers both
    long long mine = 0, before = 0;
    n.all = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        mine = b < p.a.batch ? (tiles_of<kTile, kListed>(p, b) + kUnitCost) * p.units : 0;
        n.all += scan_cta(mine, &before, scratch);
    }
    n.per = places_per_cta(n.all, ctas);
    const long long x = n.per * cta;
    long long at = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        long long sum = n.all;
        if (!once) {
            mine = b < p.a.batch ? (tiles_of<kTile, kListed>(p, b) + kUnitCost) * p.units : 0;
            sum = scan_cta(mine, &before, scratch);
        }
        const long long mine0 = at + before;
        if (entry >= 0 ? b == entry : x >= mine0 && x < mine0 + mine) {
            scratch[8] = b;
            scratch[9] = mine0;
        }
        at += sum;
    }
    __syncthreads();
    n.entry = (int)scratch[8];
    n.first = scratch[9];
    return n;
}

// Which rows of q a unit's block covers.
struct Unit {
    int b, seq, head, query, row0, len, rows;
    __device__ __forceinline__ Unit(const AttendArgs &p, bool listed, int entry, int u, int block_rows)
    {
        b = entry;
        seq = sequence_of(p, b);
        len = length_of(p, seq);
        const int block = u % p.blocks;
        u /= p.blocks;
        head = u % p.c.kv_heads;
        query = listed ? u / p.c.kv_heads : 0;
        row0 = block * block_rows;
        rows = p.rows - row0 < block_rows ? p.rows - row0 : block_rows;
    }
    // row r of the block -> (query, query head)
    __device__ __forceinline__ void row(const AttendArgs &p, int r, int *j, int *h) const
    {
        const int e = row0 + r, q = e / p.group;
        *j = query + q;
        *h = head * p.group + (e - q * p.group);
    }
};

// Query operands of a unit, the rows' factors and limits.  A row is scaled by a
// power of two to magnitudes of 2^14 to 2^15, so that fp16 holds every bf16 and
// fp16 value of it (down to 2^-39 of the largest, below which it adds nothing).
template <int D, int NT, typename T>
__device__ __forceinline__ void load_queries(const AttendArgs &p, const Unit &u, unsigned char *smem)
{
    using S = Shape<D, NT>;
    constexpr int kMine = D / 32;                  // channels of a lane
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    __half *frag = reinterpret_cast<__half *>(smem + S::kOffQ);
    float *factor = reinterpret_cast<float *>(smem + S::kOffFactor);
    int *limit = reinterpret_cast<int *>(smem + S::kOffLimit);
    for (int r = warp; r < S::kRows; r += kAttendWarps) {
        float x[kMine];
        int j = 0, h = 0;
        const bool in = r < u.rows;
        u.row(p, in ? r : 0, &j, &h);
        const T *q = (const T *)p.a.q + u.b * p.a.q_batch + j * p.a.q_query + h * p.a.q_head;
        float most = 0.f;
        bool odd = false;
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            x[e] = in ? to_float(q[lane * kMine + e]) : 0.f;
            odd |= !(fabsf(x[e]) <= 3.402823466e38f);
            most = fmaxf(most, fabsf(x[e]));
        }
#pragma unroll
        for (int step = 16; step; step /= 2)
            most = fmaxf(most, __shfl_xor_sync(~0u, most, step));
        odd = __any_sync(~0u, odd);
        int up = most > 0.f && !odd ? 14 - ((int)(__float_as_uint(most) >> 23) - 127) : 0;
        up = up > 100 ? 100 : up;
        const float lift = copysignf(__uint_as_float((unsigned)(up + 127) << 23), p.a.scale);
#pragma unroll
        for (int e = 0; e < kMine; ++e) {
            const int d = lane * kMine + e, w = d / 8, n = d % 8;
            const int group = d / kGroup, t = w % 4, half = n / 4, reg = n % 2, second = n % 4 / 2;
            frag[((((group * 2 + second) * NT + r / 8) * 32 + r % 8 * 4 + t) * 2 + reg) * 2 + half] =
                __float2half_rn(x[e] * lift * (reg ? 0.0625f : 1.f));
        }
        if (lane == 0) {
            // score in base-2 units = sum * factor, which is not negative
            factor[r] = ldexpf(fabsf(p.a.scale) * 1.4426950408889634f, -up);
            const int see = u.len - p.a.queries + 1 + j;
            limit[r] = in && see > 0 ? see : 0;
        }
    }
}

template <int D, int NT, bool kListed>
__global__ void __launch_bounds__(kAttendThreads, Shape<D, NT>::kTwoCtas ? 2 : 1)
attend_kernel(const __grid_constant__ AttendArgs p)
{
    using S = Shape<D, NT>;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
    long long *scratch = reinterpret_cast<long long *>(smem + S::kOffScan);
    unsigned char *ring = smem + warp * S::kWarpBytes;
    unsigned *masks = reinterpret_cast<unsigned *>(smem + S::kOffMask) + warp * S::kStages;
    const float *factor = reinterpret_cast<const float *>(smem + S::kOffFactor);
    const int *limit = reinterpret_cast<const int *>(smem + S::kOffLimit);
    // maximum (later weight) and sum of row r of warp w's result
    auto wmax = [&](int w, int r) -> float & {
        return *reinterpret_cast<float *>(smem + w * S::kWarpBytes + S::kOffMax + r * 4);
    };
    auto wsum = [&](int w, int r) -> float & {
        return *reinterpret_cast<float *>(smem + w * S::kWarpBytes + S::kOffSum + r * 4);
    };

    // state of the warp's ring: the stage filled and the one used next, the
    // phase of the latter; lost: a copy did not arrive, the results become NaN
    const uint32_t barriers = shared_address(smem + S::kOffBarrier) + warp * S::kStages * 8;
    int fill = 0, use = 0;
    unsigned phase = 0;
    bool lost = false;
    if (lane == 0) {
        for (int s = 0; s < S::kStages; ++s)
            barrier_init(barriers + s * 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();

    dependent_grid_wait();
    allow_dependent_grid();

    const Line line = line_of<S::kTile, kListed>(p, gridDim.x, blockIdx.x, -1, scratch);
    long long x = line.per * blockIdx.x, first = line.first;
    const long long end = x + line.per < line.all ? x + line.per : line.all;
    if (x >= end)
        return;
    int entry = line.entry;

    // Tokens of the rows of the operands: row r of a 16-token step is token
    // tok(r) of it, rows 8..15 the tokens after those of rows 0..7; an order
    // that spreads the records of a load over all banks.
    const int tok_row = g & 1 ? 8 + ((g + 3) & 7) : g;
    const int tok_a = 2 * t, tok_b = 8 + ((2 * t + 4) & 7);

    while (x < end) {
        // the part of the unit at x that is this CTA's
        const long long tiles = tiles_of<S::kTile, kListed>(p, entry), each = tiles + kUnitCost;
        const int u_in = (int)((x - first) / each);
        const long long zero = first + u_in * each + kUnitCost;    // place of the unit's tile 0
        const long long tile0 = x > zero ? x - zero : 0;
        const long long stop = zero + tiles < end ? zero + tiles : end;
        const long long count = stop - zero - tile0;
        const Unit u(p, kListed, entry, u_in, S::kRows);
        x = zero + tiles;
        if (x - first == each * p.units) {
            first = x;
            ++entry;
        }
        if (count <= 0)
            break;      // only the unit's first places: its tiles are the next CTA's

        if (p.a.bf16)
            load_queries<D, NT, __nv_bfloat16>(p, u, smem);
        else
            load_queries<D, NT, __half>(p, u, smem);

        // ---- the warp's tiles: warp, warp + 8, ... of `count` -------------
        const int mine = count > warp ? (int)((count - warp + kAttendWarps - 1) / kAttendWarps) : 0;
        const int32_t *list = kListed ? p.a.indices + ((long long)u.b * p.a.queries + u.query) * p.a.k
                                      : nullptr;
        const int seen = kListed ? u.len - p.a.queries + 1 + u.query : u.len;
        const int32_t *row_table =
            p.c.table + ((unsigned)u.seq < (unsigned)p.c.max_seqs ? u.seq * p.c.table_stride : 0);
        const unsigned char *head_pool =
            p.c.pool + (long long)u.head * p.c.page_size * S::kRecord;

        // tokens and list entries are below 2^31; the last tile may end above
        const unsigned e0 = (unsigned)((tile0 + warp) * S::kTile) + lane;
        // position of this lane's token of the warp's tile i, -1: none
        auto position = [&](int i) -> int {
            if (i >= mine || lane >= S::kTile)
                return -1;
            const unsigned e = e0 + i * (kAttendWarps * S::kTile);
            int pos = (int)e;
            if (kListed)
                pos = e < (unsigned)p.a.k ? __ldg(list + e) : -1;
            return pos < seen ? pos : -1;
        };
        auto page_of = [&](int pos) -> int {
            return pos >= 0 ? __ldg(row_table + p.by_page(pos)) : -1;
        };
        // Copies the records of a tile: a lane each, or, where `run` neighbours
        // lie side by side in a page, one lane for all of them.  A run's tokens
        // past the sequence's end are in the page too; the mask leaves them out.
        auto issue = [&](int pos, int page) {
            const uint32_t bar = barriers + fill * 8, dst = shared_address(ring + fill * S::kStageBytes);
            const bool ok = (unsigned)page < (unsigned)p.c.n_pages;   // page is -1 where pos is
            const bool leads = ok && (lane & (p.run - 1)) == 0;
            const unsigned mask = __ballot_sync(~0u, ok), leaders = __ballot_sync(~0u, leads);
            if (lane == 0) {
                masks[fill] = mask;
                barrier_expect(bar, __popc(leaders) * p.run * S::kRecord);
            }
            __syncwarp();
            if (leads) {
                const int in_page = pos - p.by_page(pos) * p.c.page_size;
                copy_bulk(dst + lane * S::kStride,
                          head_pool + page * p.c.page_stride + (long long)in_page * S::kRecord,
                          p.run * S::kRecord, bar);
            }
            fill = fill + 1 == S::kStages ? 0 : fill + 1;
        };

        // the ring held the last unit's results
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        int pos_next, page_next;
        {
            int pos[S::kStages], page[S::kStages];
#pragma unroll
            for (int s = 0; s < S::kStages; ++s)
                pos[s] = position(s);
#pragma unroll
            for (int s = 0; s < S::kStages; ++s)
                page[s] = page_of(pos[s]);
#pragma unroll
            for (int s = 0; s < S::kStages - 1; ++s) {
                if (s < mine)
                    issue(pos[s], page[s]);
            }
            pos_next = pos[S::kStages - 1];
            page_next = page[S::kStages - 1];
        }
        int pos_after = position(S::kStages);

        __syncthreads();   // query operands are there

        float o[S::kGroups][2][NT][4];
        float top[NT][2], sum[NT][2], fac[NT][2];
        int least = 0x7fffffff, lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                top[nt][c] = -INFINITY;
                sum[nt][c] = 0.f;
                fac[nt][c] = factor[nt * 8 + 2 * t + c];
                lim[nt][c] = limit[nt * 8 + 2 * t + c];
                if (nt * 8 + 2 * t + c < u.rows)
                    least = min(least, lim[nt][c]);
            }
        // tiles below the lowest limit of any row need no comparison
        least = __reduce_min_sync(~0u, least);
#pragma unroll
        for (int i = 0; i < S::kGroups; ++i)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][s][nt][e] = 0.f;

        auto consume = [&](auto masked_tag, const unsigned char *tile, unsigned mask, int base) {
            constexpr bool kMasked = decltype(masked_tag)::value;
            // scores
            float sc[S::kMT][NT][4];
#pragma unroll
            for (int mt = 0; mt < S::kMT; ++mt) {
                const unsigned char *ra = tile + (mt * 16 + tok_row) * S::kStride;
                const unsigned char *rb = ra + S::kStride;
                float sa[S::kGroups], sb[S::kGroups];
                load_scales(sa, ra + D);
                load_scales(sb, rb + D);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[mt][nt][e] = 0.f;
#pragma unroll
                for (int st = 0; st < S::kStretches; ++st) {
                    uint32_t wa[S::kPer], wb[S::kPer];
                    load_words(wa, ra + st * 64 + t * S::kPer * 4);
                    load_words(wb, rb + st * 64 + t * S::kPer * 4);
#pragma unroll
                    for (int i = 0; i < S::kPer; ++i) {
                        const int group = st * S::kPer + i;
                        const uint32_t ha = wa[i] >> 8, hb = wb[i] >> 8;
                        const uint32_t a00 = low_codes(wa[i]);
                        const uint32_t a01 = low_codes(wb[i]);
                        const uint32_t a02 = high_codes(wa[i]);
                        const uint32_t a03 = high_codes(wb[i]);
                        const uint32_t a10 = low_codes(ha);
                        const uint32_t a11 = low_codes(hb);
                        const uint32_t a12 = high_codes(ha);
                        const uint32_t a13 = high_codes(hb);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint2 *qf = reinterpret_cast<const uint2 *>(smem + S::kOffQ) +
                                              (group * 2 * NT + nt) * 32 + lane;
                            const uint2 q0 = qf[0], q1 = qf[NT * 32];
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(acc, a00, a01, a02, a03, q0.x, q0.y);
                            mma16816(acc, a10, a11, a12, a13, q1.x, q1.y);
                            sc[mt][nt][0] += sa[group] * acc[0];
                            sc[mt][nt][1] += sa[group] * acc[1];
                            sc[mt][nt][2] += sb[group] * acc[2];
                            sc[mt][nt][3] += sb[group] * acc[3];
                        }
                    }
                }
            }
            // which of the lane's tokens (step mt, row g or g + 8) rows see
            auto there = [&](int mt, int e, int nt) -> bool {
                const int token = mt * 16 + tok_row + (e >= 2);
                return (mask >> token & 1) && (kListed || base + token < lim[nt][e & 1]);
            };
            bool higher = false;
            float best[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                best[nt][0] = best[nt][1] = -INFINITY;
#pragma unroll
                for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kMasked && !there(mt, e, nt))
                            sc[mt][nt][e] = -INFINITY;
                        best[nt][e & 1] = fmaxf(best[nt][e & 1], sc[mt][nt][e]);
                    }
                higher |= best[nt][0] > top[nt][0] || best[nt][1] > top[nt][1];
            }
            // a new maximum is rare after the first tiles: only then the
            // columns' maxima are joined and the sums brought down
            if (__any_sync(~0u, higher)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float b = fmaxf(best[nt][c], top[nt][c]);
                        b = fmaxf(b, __shfl_xor_sync(~0u, b, 4));
                        b = fmaxf(b, __shfl_xor_sync(~0u, b, 8));
                        b = fmaxf(b, __shfl_xor_sync(~0u, b, 16));
                        const float down =
                            top[nt][c] == -INFINITY ? 0.f : exp2_fast((top[nt][c] - b) * fac[nt][c]);
                        top[nt][c] = b;
                        sum[nt][c] *= down;
#pragma unroll
                        for (int i = 0; i < S::kGroups; ++i)
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                o[i][s][nt][c] *= down;
                                o[i][s][nt][c + 2] *= down;
                            }
                    }
            }
            float low[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    low[nt][c] = top[nt][c] == -INFINITY ? 0.f : top[nt][c] * fac[nt][c];
            // probabilities, times the value scales, as operands; then the values
#pragma unroll
            for (int mt = 0; mt < S::kMT; ++mt) {
                const unsigned char *ra = tile + (mt * 16 + tok_row) * S::kStride;
                float sa[S::kGroups], sb[S::kGroups];
                load_scales(sa, ra + D + 2 * S::kGroups);
                load_scales(sb, ra + S::kStride + D + 2 * S::kGroups);
                float pr[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pr[nt][e] = exp2_fast(sc[mt][nt][e] * fac[nt][e & 1] - low[nt][e & 1]);
                        if (kMasked && !there(mt, e, nt))
                            pr[nt][e] = 0.f;
                        sum[nt][e & 1] += pr[nt][e];
                    }
                const unsigned char *va = tile + (mt * 16 + tok_a) * S::kStride + D / 2;
                const unsigned char *vb = tile + (mt * 16 + tok_b) * S::kStride + D / 2;
#pragma unroll
                for (int st = 0; st < S::kStretches; ++st) {
                    constexpr int kW = S::kPer / 2;
                    uint32_t wa[kW], wb[kW], xa[kW], xb[kW];
                    load_words(wa, va + st * 64 + g * kW * 4);
                    load_words(wb, vb + st * 64 + g * kW * 4);
                    load_words(xa, va + S::kStride + st * 64 + g * kW * 4);
                    load_words(xb, vb + S::kStride + st * 64 + g * kW * 4);
#pragma unroll
                    for (int i = 0; i < S::kPer; ++i) {
                        const int group = st * S::kPer + i;
                        const unsigned pick = i & 1 ? 0x7632 : 0x5410;
                        const uint32_t z = __byte_perm(wa[i / 2], wb[i / 2], pick);
                        const uint32_t y = __byte_perm(xa[i / 2], xb[i / 2], pick);
                        const uint32_t z8 = z >> 8, y8 = y >> 8;
                        const uint32_t a00 = low_codes(z);
                        const uint32_t a01 = high_codes(z);
                        const uint32_t a02 = low_codes(y);
                        const uint32_t a03 = high_codes(y);
                        const uint32_t a10 = low_codes(z8);
                        const uint32_t a11 = high_codes(z8);
                        const uint32_t a12 = low_codes(y8);
                        const uint32_t a13 = high_codes(y8);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                w[e] = pr[nt][e] * (e < 2 ? sa[group] : sb[group]);
                                if (kMasked && !there(mt, e, nt))
                                    w[e] = 0.f;   // whatever the record holds
                            }
                            const uint32_t b0 = transpose8x8(pack_half2(w[0], w[1]));
                            const uint32_t b1 = transpose8x8(pack_half2(w[2], w[3]));
                            mma16816(o[group][0][nt], a00, a01, a02, a03, b0, b1);
                            mma16816(o[group][1][nt], a10, a11, a12, a13, b0, b1);
                        }
                    }
                }
            }
        };

        for (int i = 0; i < mine; ++i) {
            // every lane is done with the stage that is filled next
            __syncwarp();
            if (i + S::kStages - 1 < mine)
                issue(pos_next, page_next);
            pos_next = pos_after;
            page_next = page_of(pos_next);
            pos_after = position(i + S::kStages + 1);

            const unsigned mask = masks[use];
            const bool came = barrier_wait(barriers + use * 8, phase);
            const unsigned char *data = ring + use * S::kStageBytes;
            if (++use == S::kStages)
                use = 0, phase ^= 1;
            if (!came)
                lost = true;
            const int base = kListed ? 0 : (int)(e0 - lane + i * (kAttendWarps * S::kTile));
            if (mask == (S::kTile == 32 ? ~0u : (1u << (S::kTile & 31)) - 1) &&
                (kListed || base + S::kTile <= least))
                consume(std::false_type{}, data, mask, base);
            else if (mask)
                consume(std::true_type{}, data, mask, base);
        }
        __syncwarp();

        // ---- the warps' results, side by side in the rings' place ----------
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float s = lost ? __int_as_float(0x7fffffff) : sum[nt][c];
                s += __shfl_xor_sync(~0u, s, 4);
                s += __shfl_xor_sync(~0u, s, 8);
                s += __shfl_xor_sync(~0u, s, 16);
                const int r = nt * 8 + 2 * t + c;
                if (g == 0) {
                    wmax(warp, r) = top[nt][c] == -INFINITY ? -INFINITY : top[nt][c] * fac[nt][c];
                    wsum(warp, r) = s;
                }
                float *dst = reinterpret_cast<float *>(ring) + r * S::kOutStride + 4 * g;
#pragma unroll
                for (int i = 0; i < S::kGroups; ++i)
                    *reinterpret_cast<float4 *>(dst + i * kGroup) =
                        make_float4(o[i][0][nt][c], o[i][0][nt][c + 2] * 0.0625f,
                                    o[i][1][nt][c], o[i][1][nt][c + 2] * 0.0625f);
            }
        __syncthreads();

        const bool whole = count == tiles;
        float *part = p.a.partial + (blockIdx.x * 2LL + (tile0 == 0)) * S::kPartial;
        // weights of the warps' results: 2^(max - largest max)
        if (threadIdx.x < S::kRows) {
            const int r = threadIdx.x;
            float m = -INFINITY, l = 0.f;
            for (int w = 0; w < kAttendWarps; ++w)
                m = fmaxf(m, wmax(w, r));
            for (int w = 0; w < kAttendWarps; ++w) {
                const float f = wmax(w, r);
                // a warp that saw nothing has sum 0; one whose scores are NaN
                // has a maximum of -inf, and its NaN goes on
                const float weight = m == -INFINITY ? 1.f : exp2_fast(f - m);
                const float s = wsum(w, r);
                l += s == 0.f ? 0.f : s * weight;
                wmax(w, r) = s != s ? 1.f : weight;
            }
            if (whole) {
                wsum(0, r) = l == 0.f ? 0.f : 1.f / l;
                if (r < u.rows && p.a.lse) {
                    int j, h;
                    u.row(p, r, &j, &h);
                    p.a.lse[((long long)u.b * p.a.queries + j) * p.a.heads + h] =
                        l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
            } else {
                part[r] = m;
                part[S::kRows + r] = l;
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < S::kRows * D / 4; e += kAttendThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            if (r >= u.rows)
                break;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kAttendWarps; ++w) {
                const float4 f = *reinterpret_cast<const float4 *>(
                    smem + w * S::kWarpBytes + (r * S::kOutStride + d) * 4);
                const float weight = wmax(w, r);
                v.x += f.x * weight, v.y += f.y * weight, v.z += f.z * weight, v.w += f.w * weight;
            }
            if (whole) {
                const float inv = wsum(0, r);
                int j, h;
                u.row(p, r, &j, &h);
                const long long to = (((long long)u.b * p.a.queries + j) * p.a.heads + h) * D + d;
                if (p.a.bf16) {
                    __nv_bfloat16 y[4];
                    from_float(y[0], v.x * inv), from_float(y[1], v.y * inv);
                    from_float(y[2], v.z * inv), from_float(y[3], v.w * inv);
                    *reinterpret_cast<uint2 *>((__nv_bfloat16 *)p.a.out + to) =
                        *reinterpret_cast<const uint2 *>(y);
                } else {
                    __half y[4];
                    from_float(y[0], v.x * inv), from_float(y[1], v.y * inv);
                    from_float(y[2], v.z * inv), from_float(y[3], v.w * inv);
                    *reinterpret_cast<uint2 *>((__half *)p.a.out + to) =
                        *reinterpret_cast<const uint2 *>(y);
                }
            } else {
                *reinterpret_cast<float4 *>(part + 2 * S::kRows + r * D + d) = v;
            }
        }
        __syncthreads();
    }
}

// Joins the partial results of units that several CTAs worked on: one warp a
// query row, CTAs' shares in order.
template <int D, int NT, bool kListed>
__global__ void __launch_bounds__(kAttendThreads)
join_kernel(const __grid_constant__ AttendArgs p, int ctas)
{
    using S = Shape<D, NT>;
    __shared__ long long scratch[16];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    // blocks of 8 rows of a unit
    const long long unit = blockIdx.x / NT;
    const int u_in = (int)(unit % p.units);
    const Line line = line_of<S::kTile, kListed>(p, ctas, 0, (int)(unit / p.units), scratch);
    const int entry = line.entry;
    const long long per = line.per, tiles = tiles_of<S::kTile, kListed>(p, entry);
    const long long from = line.first + u_in * (tiles + kUnitCost) + kUnitCost;
    const long long c0 = from / per, c1 = (from + tiles - 1) / per;
    const int r = blockIdx.x % NT * 8 + warp;
    const Unit u(p, kListed, entry, u_in, S::kRows);
    if (c0 == c1 || r >= u.rows)
        return;
    // Up to here only what the launch before the attention left is read: this
    // launch starts when that one has been waited for.
    dependent_grid_wait();
    // a CTA's second place holds the unit that begins in it
    auto place = [&](long long c) { return p.a.partial + (c * 2 + (c == c0)) * S::kPartial; };
    float m = -INFINITY;
    for (long long c = c0 + lane; c <= c1; c += 32)
        m = fmaxf(m, place(c)[r]);
#pragma unroll
    for (int step = 16; step; step /= 2)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, step));
    const float low = m == -INFINITY ? 0.f : m;
    float l = 0.f, v[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        v[i] = 0.f;
#pragma unroll 4
    for (long long c = c0; c <= c1; ++c) {
        const float *q = place(c);
        const float s = q[S::kRows + r];
        const float weight = s != s ? 1.f : exp2_fast(q[r] - low);
        l += s * weight;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            v[i] += q[2 * S::kRows + r * D + i * 32 + lane] * weight;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    int j, h;
    u.row(p, r, &j, &h);
    const long long row = ((long long)u.b * p.a.queries + j) * p.a.heads + h;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
        if (p.a.bf16)
            from_float(((__nv_bfloat16 *)p.a.out)[row * D + i * 32 + lane], v[i] * inv);
        else
            from_float(((__half *)p.a.out)[row * D + i * 32 + lane], v[i] * inv);
    }
    if (p.a.lse && lane == 0)
        p.a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ---- host ----------------------------------------------------------------------
// Columns of eight rows that a unit works on at once: as many as its rows
// fill, up to 4 (2 for D = 256, whose outputs would not fit the registers).
template <int D>
int row_tiles(int rows)
{
    return rows <= 8 ? 1 : rows <= 16 || D == 256 ? 2 : 4;
}

template <int D, int NT>
int attend_grid(int sms)
{
    return sms * (Shape<D, NT>::kTwoCtas ? 2 : 1);
}

template <int D, int NT, bool kListed>
cudaError_t launch_shape(AttendArgs &p, int sms, cudaStream_t stream)
{
    using S = Shape<D, NT>;
    const int ctas = attend_grid<D, NT>(sms);
    p.blocks = (p.rows + S::kRows - 1) / S::kRows;
    p.units = p.c.kv_heads * p.blocks * (kListed ? p.a.queries : 1);
    p.sel_tiles = ((long long)p.a.k + S::kTile - 1) / S::kTile;
    auto fn = attend_kernel<D, NT, kListed>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(kAttendThreads);
    cfg.dynamicSmemBytes = S::kSmem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if ((e = cudaLaunchKernelEx(&cfg, fn, (const AttendArgs)p)) != cudaSuccess)
        return e;
    cfg.gridDim = dim3((unsigned)((long long)p.a.batch * p.units * NT));
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join_kernel<D, NT, kListed>, (const AttendArgs)p, ctas);
}

template <int D>
cudaError_t launch_dim(const Cache &c, const Attend &a, int sms, cudaStream_t stream)
{
    AttendArgs p;
    p.c = c;
    p.a = a;
    p.by_page.set(c.page_size);
    p.group = a.heads / c.kv_heads;
    p.run = 1;
    if (!a.indices && Shape<D, 1>::kStride == Shape<D, 1>::kRecord)
        while (p.run < Shape<D, 1>::kTile && c.page_size % (2 * p.run) == 0)
            p.run *= 2;
    p.rows = a.indices ? p.group : p.group * a.queries;
    const int nt = row_tiles<D>(p.rows);
    if (a.indices)
        return nt == 1   ? launch_shape<D, 1, true>(p, sms, stream)
               : nt == 2 ? launch_shape<D, 2, true>(p, sms, stream)
                         : launch_shape<D, D == 256 ? 2 : 4, true>(p, sms, stream);
    return nt == 1   ? launch_shape<D, 1, false>(p, sms, stream)
           : nt == 2 ? launch_shape<D, 2, false>(p, sms, stream)
                     : launch_shape<D, D == 256 ? 2 : 4, false>(p, sms, stream);
}

template <int D>
size_t workspace_dim(int rows, int sms)
{
    const int nt = row_tiles<D>(rows);
    const size_t floats = nt == 1   ? (size_t)attend_grid<D, 1>(sms) * Shape<D, 1>::kPartial
                          : nt == 2 ? (size_t)attend_grid<D, 2>(sms) * Shape<D, 2>::kPartial
                                    : (size_t)attend_grid<D, D == 256 ? 2 : 4>(sms) *
                                          Shape<D, D == 256 ? 2 : 4>::kPartial;
    return 2 * floats * sizeof(float);
}

}  // namespace kv4
}  // namespace ds
