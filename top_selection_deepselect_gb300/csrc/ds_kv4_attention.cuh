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
// A unit is up to kRows (query, head) rows that share a key/value head.  With 8
// rows the matrix instructions (m16n8k16) have tokens or channels as their 16
// rows and the query rows as their 8 columns:
//   S^T = K Q^T,  O^T = V^T P^T
// and P is transposed between the two by a movmatrix per 8 x 8.  With 16 rows
// (grouped heads, drafted tokens) the query rows are the 16 rows instead,
//   S = Q K^T,  O = P V
// which is twice the products from the same expanded codes, and P comes out as it
// goes in.  Either way the sum over each group of 32 channels is multiplied by the key
// scale of (token, group) in 32 bits, and the probabilities carry the value
// scale, fp16(p * scale), the only rounding of the inner loop; 32-bit operands
// would halve the rate of the matrix instructions.  Scales reach from 2^-24 to
// 2^16, so a power of two goes with each weight: p is taken 2^23 times, and
// each warp lifts the scales of a group so that the largest it has met comes to
// lie in [2^-9, 2^-8).  Weights are then below 2^15 and keep 11 significant bits,
// 2^-11 relative, while p * scale is above 2^-28 of the group's largest scale
// (times the largest p); below, they are off by 2^-39 of it at most.  Lifts only
// fall while a warp goes through a unit; the output is brought down with them,
// and they are taken back at the unit's end.  Denominators are summed in 32 bits
// from unrounded p.
//
// Work is cut into tiles of kTile tokens; all tiles of all (sequence, head)
// units stand in one line that is divided evenly among the CTAs, whatever the
// lengths are; they are read on the device, so that the host needs to know
// nothing.  A CTA's warps take its tiles in turn, each with its own ring of
// asynchronous copies, running maximum, sum and output, and meet only at the
// end of a unit.  A unit cut between CTAs leaves partial results in the
// workspace; a second launch joins them in a fixed order.
#pragma once

#include <atomic>
#include <cooperative_groups.h>
#include <type_traits>

#include "ds_device.cuh"
#include "ds_host.h"
#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {

// Shape of one instantiation: head dimension, query rows of a unit (8 or 16).
template <int D, int Rows>
struct Shape {
    static constexpr bool kWide = Rows > 8;                      // query rows are the operands' rows
    static constexpr int kRows = Rows;
    static constexpr int kSubs = kWide ? 4 : 2;                  // instructions of a group's values
    static constexpr int kGroups = D / kGroup;
    static constexpr int kStretches = D > 128 ? D / 128 : 1;    // of up to 128 channels
    static constexpr int kPer = kGroups / kStretches;            // groups of a stretch
    static constexpr int kMT = D == 256 ? 1 : 2;                 // 16-token steps of a tile
    static constexpr int kTile = 16 * kMT;
    static constexpr unsigned kFullMask = ~0u >> (32 - kTile);
    static constexpr int kRecord = record_bytes(D);
    static constexpr int kStageBytes = kTile * kRecord;
    static constexpr int kOutRegs = kGroups * kSubs * 4;
    // Warps of a CTA and CTAs of an SM, by what the output leaves of the
    // registers: 2 x 8 warps with 128 each, 12 with 168, 8 with 255.  (16 warps
    // in one CTA, both timed before scales were lifted: 64 x 32768 tokens the same
    // 403 us, 256 x 200 tokens 63 for 41, because nothing else runs while a unit
    // ends.)
    static constexpr int kWarps = kOutRegs == 64 ? 12 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kCtas = kOutRegs <= 32 ? 2 : 1;
    static constexpr int kStages = D == 64 ? (kCtas == 2 ? 4 : 6) : kCtas == 2 ? 3 : kWarps == 12 ? 4 : 5;
    static constexpr int kOutStride = D + 4;                     // floats of an output row in shared memory
    // A warp's ring; at a unit's end its tail holds the warp's output, the rows'
    // maxima and sums, while kEarly stages in front of that are filled for the
    // next unit.
    static constexpr int kResultBytes = kRows * (kOutStride + 2) * 4;
    static constexpr int kWarpBytes =
        kStages * kStageBytes > kResultBytes ? kStages * kStageBytes : kResultBytes;
    static constexpr int kTail = kWarpBytes - kResultBytes;
    static constexpr int kOffMax = kTail + kRows * kOutStride * 4;
    static constexpr int kOffSum = kOffMax + kRows * 4;
    static constexpr int kEarly =
        kTail / kStageBytes < kStages - 1 ? kTail / kStageBytes : kStages - 1;
    // shared memory behind the rings
    static constexpr int kOffQ = kWarps * kWarpBytes;             // query operands
    static constexpr int kOffFactor = kOffQ + kRows * D * 2;
    static constexpr int kOffLimit = kOffFactor + kRows * 4;
    static constexpr int kOffBarrier = (kOffLimit + kRows * 4 + 15) / 16 * 16;
    static constexpr int kOffMask = kOffBarrier + kWarps * kStages * 8;
    static constexpr int kOffScan = (kOffMask + kWarps * kStages * 4 + 15) / 16 * 16;
    static constexpr int kOffPart = kOffScan + 16 * 8;
    // a warp's value scales, two groups a word: the largest that its lifts are
    // good for, and the lifts
    static constexpr int kOffBound = kOffPart + 2 * 128;
    static constexpr int kOffLift = kOffBound + kWarps * kGroups * 2;
    static constexpr int kSmem = kOffLift + kWarps * kGroups * 2;
    static_assert(kSmem <= (kCtas == 2 ? 115712 : 232448), "shared memory of an SM");
    static constexpr int kPartial = kRows * (D + 2);                    // floats of a partial result

    // Order of the 16 tokens of a step in the operands: places 2 t and 2 t + 1
    // (t < 4) hold tokens even(t) and odd(t), places 8 above hold the tokens
    // kNext after those.  With records of 80, 144 and 288 bytes the operand
    // loads of a warp then touch every bank equally often.
    static constexpr int kNext = D == 256 ? 8 : 1;
    static __device__ __forceinline__ int even(int t) { return D == 256 ? t : 2 * t; }
    static __device__ __forceinline__ int odd(int t)
    {
        return D == 256 ? 4 + ((t + 2) & 3) : 8 + ((2 * t + 4) & 7);
    }
};

struct AttendArgs {
    Cache c;
    Attend a;
    long long sel_tiles;  // tiles of a unit when tokens are listed
    long long parts;      // floats of the workspace before the partial results
    int run;              // tokens of a tile that lie side by side in a page, a power of two
    int group;            // query heads of a key/value head
    int rows;             // query rows of a unit before it is cut into blocks
    int blocks;           // blocks of kRows rows, a unit each
    int units;            // units of a batch entry
    int whole;            // units are not cut: each is its first place's CTA's
    int cluster;          // > 1: a unit is a cluster's, cut evenly and joined in it
    Divider by_group, by_blocks, by_heads;
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

// Nanoseconds that a copy is waited for, far beyond any copy's time: one that
// never ends must not hang the GPU.
constexpr long long kPatience = 1000000000;
__device__ __forceinline__ bool barrier_done(uint32_t bar, unsigned phase)
{
    unsigned done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(phase) : "memory");
    return done != 0;
}

__device__ __forceinline__ long long nanoseconds()
{
    long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Waits for a phase to end.  late: this lane has given a phase up, now or before,
// and waits for none any more.  Other lanes may not have, so that no branch that
// leads away from them is taken on it.
__device__ __forceinline__ void barrier_wait(uint32_t bar, unsigned phase, bool &late,
                                             long long patience = kPatience)
{
    if (barrier_done(bar, phase) || late)
        return;
    const long long from = nanoseconds();
    while (!barrier_done(bar, phase))
        if (nanoseconds() - from > patience) {
            late = true;
            return;
        }
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

// Lift of a group whose largest value scale has the bits `most` (a float, not 0):
// the power of two that brings it to [2^-9, 2^-8), in fp16; weights are made of
// probabilities times kRaise.  What that makes the output too large by, inverted.
constexpr float kRaise = 0x1p23f;
__device__ __forceinline__ unsigned lift_of(unsigned most)
{
    return __half_as_ushort(__float2half_rn(__uint_as_float((245u - (most >> 23)) << 23)));
}
__device__ __forceinline__ float lift_back(unsigned lift)
{
    const float f = __half2float(__ushort_as_half((unsigned short)lift));
    return __uint_as_float((254u << 23) - __float_as_uint(f)) * (1.f / kRaise);
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

template <int N>
__device__ __forceinline__ void store_words(unsigned char *p, const uint32_t (&w)[N])
{
#pragma unroll
    for (int i = 0; i < N; ++i)
        reinterpret_cast<uint32_t *>(p)[i] = w[i];
}

template <typename T>
__device__ __forceinline__ void store_four(T *dst, const float4 &v, float factor)
{
    T y[4];
    from_float(y[0], v.x * factor), from_float(y[1], v.y * factor);
    from_float(y[2], v.z * factor), from_float(y[3], v.w * factor);
    *reinterpret_cast<uint2 *>(dst) = *reinterpret_cast<const uint2 *>(y);
}

// Scales of G groups, each times its lift, as floats: the product of two fp16
// numbers is exact there.
template <int G>
__device__ __forceinline__ void load_lifted(float (&s)[G], const unsigned char *p,
                                            const uint32_t (&lift)[G / 2])
{
    uint32_t w[G / 2];
    load_words(w, p);
#pragma unroll
    for (int i = 0; i < G / 2; ++i)
        asm("{\n\t.reg .b16 x, y, f, g;\n\t"
            "mov.b32 {x, y}, %2;\n\t"
            "mov.b32 {f, g}, %3;\n\t"
            "fma.rn.f32.f16 %0, x, f, %4;\n\t"
            "fma.rn.f32.f16 %1, y, g, %4;\n\t}"
            : "=f"(s[2 * i]), "=f"(s[2 * i + 1])
            : "r"(w[i]), "r"(lift[i]), "f"(-0.f));
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
    return p.a.seqs ? p.a.seqs[b] : b;
}

__device__ __forceinline__ int length_of(const AttendArgs &p, int seq)
{
    if ((unsigned)seq >= (unsigned)p.c.max_seqs)
        return 0;
    const int n = p.a.lengths[seq];
    const long long room = (long long)p.c.max_pages * p.c.page_size;
    return n < 0 ? 0 : n > room ? (int)room : n;
}

// Tiles of every unit of batch entry b: at least one, so that rows that see
// nothing are written too.
template <int kTile>
__device__ __forceinline__ long long tiles_of(const AttendArgs &p, bool listed, int b)
{
    if (listed)
        return p.sel_tiles;
    const int n = length_of(p, sequence_of(p, b));
    return n > kTile ? (n + kTile - 1LL) / kTile : 1;
}

// Sum over the CTA, and in *before the sum of the threads below.
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
// places the CTA that meets 24 empty sequences in a row takes three times as long
// as the others (37 ragged sequences of 5 drafts: 84 us; with 12, 18, 24, 32 and 40
// places 37, 35, 33 to 35, 35 and 37; 16 x 16384 tokens 70 with any of them).
constexpr int kUnitCost = 24;

// Quotient of numbers that are not negative, in 32 bits where that is enough.
__device__ __forceinline__ long long divided(long long a, long long b)
{
    return (a | b) >> 32 == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Places of the line for each CTA: two tiles a warp at least where units are
// cut, so that there are not more parts to join than the work is worth.
__device__ __forceinline__ long long places_per_cta(const AttendArgs &p, long long all)
{
    const long long even = divided(all + gridDim.x - 1, gridDim.x);
    const int least = p.whole ? 1 : 2 * (blockDim.x / 32);
    return even > least ? even : least;
}

// The line's length, places for each CTA, and the batch entry that this CTA's
// first place belongs to with the entry's own first place.
struct Line {
    long long all, per, first;
    int entry;
};

template <int kTile>
__device__ __forceinline__ Line line_of(const AttendArgs &p, bool listed, long long *scratch)
{
    Line n;
    if (listed) {
        const long long each = (p.sel_tiles + kUnitCost) * p.units;
        n.all = each * p.a.batch;
        n.per = places_per_cta(p, n.all);
        n.entry = (int)divided(n.per * blockIdx.x, each);
        n.first = n.entry * each;
        return n;
    }
    const bool once = p.a.batch <= (int)blockDim.x;   // then one scan answers both
    long long mine = 0, before = 0;
    n.all = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        mine = b < p.a.batch ? (tiles_of<kTile>(p, listed, b) + kUnitCost) * p.units : 0;
        n.all += scan_cta(mine, &before, scratch);
    }
    n.per = places_per_cta(p, n.all);
    const long long x = n.per * blockIdx.x;
    long long at = 0;
    for (int b0 = 0; b0 < p.a.batch; b0 += blockDim.x) {
        const int b = b0 + threadIdx.x;
        long long sum = n.all;
        if (!once) {
            mine = b < p.a.batch ? (tiles_of<kTile>(p, listed, b) + kUnitCost) * p.units : 0;
            sum = scan_cta(mine, &before, scratch);
        }
        if (x >= at + before && x < at + before + mine) {
            scratch[14] = b;
            scratch[15] = at + before;
        }
        at += sum;
    }
    __syncthreads();
    n.entry = (int)scratch[14];
    n.first = scratch[15];
    return n;
}

// Which query rows unit u of a batch entry covers.
struct Unit {
    int b = 0, head = 0, query = 0, row0 = 0, rows = 0;
    Unit() = default;
    __device__ __forceinline__ Unit(const AttendArgs &p, int entry, int u, int block_rows)
    {
        b = entry;
        const int v = p.by_blocks(u), block = u - v * p.blocks, q = p.by_heads(v);
        head = v - q * p.c.kv_heads;
        query = q;    // 0 unless tokens are listed: then each query is a unit of its own
        row0 = block * block_rows;
        rows = p.rows - row0 < block_rows ? p.rows - row0 : block_rows;
    }
    // row r of the block -> (query, query head)
    __device__ __forceinline__ void row(const AttendArgs &p, int r, int *j, int *h) const
    {
        const int e = row0 + r, q = p.by_group(e);
        *j = query + q;
        *h = head * p.group + (e - q * p.group);
    }
};

// What a CTA works on, kept in shared memory so that the loop over tiles has
// the registers for itself.
struct Part {
    const int32_t *list, *row_table;     // listed positions; the sequence's row of the table
    const unsigned char *head_pool;      // records of the head in page 0
    long long next;                      // place of the line where the next unit begins
    Unit u;
    int next_entry, next_unit;           // and which one it is
    int seen;                            // positions attended are below `seen`
    int whole, begins, active;           // all of the unit's tiles are this CTA's; its first one is;
                                         // warps that have tiles
};
static_assert(sizeof(Part) <= 128, "room in Shape");

// Left for the join: the unit that begins in a CTA and goes on in others.
struct alignas(16) Split {
    int b, unit, parts, pad;
};

// Query operands of a unit, the rows' factors and limits.  A row is scaled by a
// power of two to magnitudes of 2^14 to 2^15, so that fp16 holds every bf16 and
// fp16 value of it down to 2^-25 of the largest; smaller ones are off by 2^-35 of
// that at most.
template <int D, int Rows>
struct Queries {
    using S = Shape<D, Rows>;
    static constexpr int kMine = D / 32;                                    // channels of a lane
    static constexpr int kTurns = (Rows + S::kWarps - 1) / S::kWarps;       // rows of a warp
    float x[kTurns][kMine] = {};

    template <typename T>
    __device__ __forceinline__ void load(const AttendArgs &p, const Unit &u)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = warp + i * S::kWarps;
            const bool in = r < u.rows;
            int j = 0, h = 0;
            u.row(p, in ? r : 0, &j, &h);
            const T *q = (const T *)p.a.q + u.b * p.a.q_batch + j * p.a.q_query + h * p.a.q_head;
#pragma unroll
            for (int e = 0; e < kMine; ++e)
                x[i][e] = in ? to_float(q[lane * kMine + e]) : 0.f;
        }
    }

    __device__ __forceinline__ void load(const AttendArgs &p, const Unit &u)
    {
        if (p.a.bf16)
            load<__nv_bfloat16>(p, u);
        else
            load<__half>(p, u);
    }

    __device__ __forceinline__ void store(const AttendArgs &p, const Unit &u, int len, unsigned char *smem)
    {
        const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
        __half *frag = reinterpret_cast<__half *>(smem + S::kOffQ);
        float *factor = reinterpret_cast<float *>(smem + S::kOffFactor);
        int *limit = reinterpret_cast<int *>(smem + S::kOffLimit);
#pragma unroll
        for (int i = 0; i < kTurns; ++i) {
            const int r = warp + i * S::kWarps;
            if (r >= Rows)
                break;
            // the bits of magnitudes are in the magnitudes' order, those that
            // are not finite above all others
            unsigned most = 0;
#pragma unroll
            for (int e = 0; e < kMine; ++e)
                most = max(most, __float_as_uint(x[i][e]) & 0x7fffffffu);
            most = __reduce_max_sync(~0u, most);
            int up = most > 0 && most < 0x7f800000u ? 14 + 127 - (int)(most >> 23) : 0;
            up = up > 100 ? 100 : up;
            const float lift = copysignf(__uint_as_float((unsigned)(up + 127) << 23), p.a.scale);
#pragma unroll
            for (int e = 0; e < kMine; ++e) {
                const int d = lane * kMine + e, w = d / 8, n = d % 8;
                const int group = d / kGroup, t = w % 4, half = n / 4, reg = n % 2, second = n % 4 / 2;
                // operand register of the lane that holds row r % 8, place 2 t:
                // narrow {reg}, wide {reg, row / 8}
                const int at = S::kWide ? ((group * 2 + second) * 32 + r % 8 * 4 + t) * 4 +
                                              reg * 2 + r / 8
                                        : ((group * 2 + second) * 32 + r * 4 + t) * 2 + reg;
                frag[at * 2 + half] = __float2half_rn(x[i][e] * lift * (reg ? 0.0625f : 1.f));
            }
            if (lane == 0) {
                // score in base-2 units = sum * factor, which is not negative;
                // 2^-up in two steps, each of them a normal number
                const float down = __uint_as_float((unsigned)(127 - up / 2) << 23) *
                                   (fabsf(p.a.scale) * 1.4426950408889634f);
                factor[r] = down * __uint_as_float((unsigned)(127 - (up - up / 2)) << 23);
                int j, h;
                u.row(p, r < u.rows ? r : 0, &j, &h);
                const int see = len - p.a.queries + 1 + j;
                limit[r] = r < u.rows && see > 0 ? see : 0;
            }
        }
    }
};

// kRun: every token is attended and pages hold whole runs of this many tokens,
// a tile or half of one; 0: tokens are looked up one by one, listed or not.
template <int D, int Rows, int kRun>
__global__ void __launch_bounds__((Shape<D, Rows>::kThreads), (Shape<D, Rows>::kCtas))
attend_kernel(const __grid_constant__ AttendArgs p)
{
    using S = Shape<D, Rows>;
    const bool listed = kRun == 0 && p.a.indices != nullptr;
    extern __shared__ __align__(128) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
    long long *scratch = reinterpret_cast<long long *>(smem + S::kOffScan);
    unsigned char *ring = smem + warp * S::kWarpBytes;
    unsigned *masks = reinterpret_cast<unsigned *>(smem + S::kOffMask) + warp * S::kStages;
    const float *factor = reinterpret_cast<const float *>(smem + S::kOffFactor);
    const int *limit = reinterpret_cast<const int *>(smem + S::kOffLimit);
    unsigned char *bounds = smem + S::kOffBound + warp * S::kGroups * 2;
    unsigned char *lifts = smem + S::kOffLift + warp * S::kGroups * 2;
    // maximum (later weight) and sum of row r of warp w's result
    auto wmax = [&](int w, int r) -> float & {
        return *reinterpret_cast<float *>(smem + w * S::kWarpBytes + S::kOffMax + r * 4);
    };
    auto wsum = [&](int w, int r) -> float & {
        return *reinterpret_cast<float *>(smem + w * S::kWarpBytes + S::kOffSum + r * 4);
    };

    // state of the warp's ring: tile i of a unit is in stage i % kStages; the
    // stage filled and the one used next, the phases of all; lost: a copy did not
    // arrive, the ring is not used any more and all further results are NaN; late:
    // so far only this lane knows, and starts no copies
    const uint32_t barriers = shared_address(smem + S::kOffBarrier) + warp * S::kStages * 8;
    int fill = 0, use = 0;
    unsigned phases = 0;
    bool lost = false, late = false;
    if (lane == 0) {
        for (int s = 0; s < S::kStages; ++s)
            barrier_init(barriers + s * 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();

    dependent_grid_wait();
    allow_dependent_grid();

    Split *split = reinterpret_cast<Split *>(p.a.partial) + blockIdx.x;
    const bool clustered = kRun == 0 && p.cluster > 1;
    if (threadIdx.x == 0 && !p.whole && !clustered)
        split->parts = 0;

    // place to go on at, the unit there (number u_in of its entry) and where it begins
    long long x, per, end, start;
    int entry, u_in;
    if (clustered) {
        const int n = blockIdx.x / p.cluster, rank = blockIdx.x % p.cluster;
        entry = n / p.units;
        u_in = n - entry * p.units;
        start = per = 0;
        x = kUnitCost + p.sel_tiles * rank / p.cluster;
        end = kUnitCost + p.sel_tiles * (rank + 1) / p.cluster;
    } else {
        const Line line = line_of<S::kTile>(p, listed, scratch);
        per = line.per;
        x = per * blockIdx.x;
        end = x + per < line.all ? x + per : line.all;
        if (x >= end)
            return;
        entry = line.entry;
        const long long each = tiles_of<S::kTile>(p, listed, entry) + kUnitCost;
        u_in = (int)divided(x - line.first, each);
        start = line.first + u_in * each;
        if (p.whole && x > start) {
            x = start = start + each;
            if (++u_in == p.units)
                u_in = 0, ++entry;
            if (x >= end)
                return;
        }
    }

    const int tok_row = g & 1 ? S::odd(g / 2) : S::even(g / 2);   // token at place g
    const int tok_a = S::even(t), tok_b = S::odd(t);              // at places 2 t and 2 t + 1

    // ---- the next unit: what it is, its first copies ---------------------
    int mine = 0, slot = 0;       // the warp's tiles; which `Part` is the unit's
    unsigned e0 = 0;              // first token, or list entry, of the first of them
    Part now;
    Unit unit;
    int len = 0;
    long long tiles = 0, zero = 0, tile0 = 0, count = 0;
    Queries<D, Rows> queries;
    auto part_of = [&](int i) -> volatile Part & {
        return *reinterpret_cast<Part *>(smem + S::kOffPart + i * 128);
    };

    // ---- tokens one by one: a lane each -----------------------------
    // position of this lane's token of the warp's tile i, -1: none
    auto position = [&](const volatile Part &part, int i) -> int {
        if (i >= mine || lane >= S::kTile)
            return -1;
        const unsigned e = e0 + lane + i * (S::kWarps * S::kTile);
        int pos = (int)e;
        if (listed)
            pos = e < (unsigned)p.a.k ? part.list[e] : -1;
        return pos < part.seen ? pos : -1;
    };
    auto page_of = [&](const volatile Part &part, int pos) -> int {
        return pos >= 0 ? part.row_table[p.c.by_page(pos)] : -1;
    };
    // Copies the records of a tile: a lane each, or, where `run` neighbours
    // lie side by side in a page, one lane for all of them.  A run's tokens
    // past the sequence's end are in the page too; the mask leaves them out.
    auto issue_tokens = [&](const volatile Part &part, int pos, int page) {
        const uint32_t bar = barriers + fill * 8, dst = shared_address(ring + fill * S::kStageBytes);
        const bool ok = (unsigned)page < (unsigned)p.c.n_pages;   // page is -1 where pos is
        const bool leads = ok && (lane & (p.run - 1)) == 0 && !late;
        const unsigned mask = __ballot_sync(~0u, ok), leaders = __ballot_sync(~0u, leads);
        if (lane == 0 && !late) {
            masks[fill] = mask;
            barrier_expect(bar, __popc(leaders) * p.run * S::kRecord);
        }
        __syncwarp();
        if (leads) {
            const int in_page = pos - p.c.by_page(pos) * p.c.page_size;
            copy_bulk(dst + lane * S::kRecord,
                      part.head_pool + page * p.c.page_stride + (long long)in_page * S::kRecord,
                      p.run * S::kRecord, bar);
        }
        fill = fill + 1 == S::kStages ? 0 : fill + 1;
    };
    // ---- runs: a lane looks up one of 32 whole runs ------------------
    // Tile i is run(s) i << halves and the next; 32 runs are looked up at once.
    constexpr int halves = kRun > 0 && kRun < S::kTile ? 1 : 0, per_look = 32 >> halves;
    const unsigned char *run_src = nullptr;    // of the lane's run of those under way
    unsigned tile_mask = 0;                    // of the run's tile
    int run_page = -1;                         // of the lane's run of the next ones
    auto run_pos = [&](int i0) {
        return (int)(e0 + (i0 + (lane >> halves)) * (S::kWarps * S::kTile) + (lane & halves) * kRun);
    };
    auto run_page_of = [&](const volatile Part &part, int i0) -> int {
        const int pos = run_pos(i0);
        return i0 + (lane >> halves) < mine && (unsigned)pos < (unsigned)part.seen
                   ? part.row_table[p.c.by_page(pos)] : -1;
    };
    auto next_runs = [&](const volatile Part &part, int i0) {
        const int pos = run_pos(i0);
        const bool ok = (unsigned)run_page < (unsigned)p.c.n_pages;
        const int in_page = ok ? pos - p.c.by_page(pos) * p.c.page_size : 0;
        run_src = ok ? part.head_pool + run_page * p.c.page_stride + (long long)in_page * S::kRecord
                     : nullptr;
        const int left = part.seen - pos;      // > 0 where there is a page
        tile_mask = !ok ? 0u : ~0u >> (32 - (left < kRun ? left : kRun));
        if (halves) {
            tile_mask <<= (lane & 1) * 16;
            tile_mask |= __shfl_xor_sync(~0u, tile_mask, 1);
        }
        run_page = run_page_of(part, i0 + per_look);
    };
    // tokens past the sequence's end are in the page too
    auto issue_runs = [&](const volatile Part &part, int i) {
        const int turn = i & (per_look - 1);
        if (i > 0 && turn == 0)
            next_runs(part, i);
        const uint32_t bar = barriers + fill * 8;
        if (lane == turn << halves && !late) {
            masks[fill] = tile_mask;
            const int runs = !halves ? tile_mask != 0 : ((tile_mask & 0xffffu) != 0) + (tile_mask > 0xffffu);
            barrier_expect(bar, runs * kRun * S::kRecord);
        }
        if (halves)
            __syncwarp();
        if (lane >> halves == turn && run_src && !late)
            copy_bulk(shared_address(ring + fill * S::kStageBytes) + (lane & halves) * kRun * S::kRecord,
                      run_src, kRun * S::kRecord, bar);
        fill = fill + 1 == S::kStages ? 0 : fill + 1;
    };

    // The part of the unit at x that is this CTA's: looks its first tiles up,
    // starts kEarly copies and the load of its queries.  False: there is none.
    int pos_next = -1, page_next = -1, pos_after = -1;
    int early_pos[S::kStages], early_page[S::kStages];
    auto set_up = [&]() -> bool {
        // nothing of the last unit is carried through the loop over its tiles
        now = Part();
        unit = Unit();
        queries = Queries<D, Rows>();
        len = mine = 0;
        tiles = zero = tile0 = count = 0;
        e0 = tile_mask = 0;
        run_src = nullptr;
        run_page = pos_next = page_next = pos_after = -1;
#pragma unroll
        for (int s = 0; s < S::kStages; ++s)
            early_pos[s] = early_page[s] = -1;
        if (x >= end)
            return false;
        const int seq = sequence_of(p, entry);
        len = length_of(p, seq);
        tiles = tiles_of<S::kTile>(p, listed, entry);
        zero = start + kUnitCost;     // place of the unit's tile 0
        tile0 = x > zero ? x - zero : 0;
        const long long stop = p.whole || zero + tiles < end ? zero + tiles : end;
        count = stop - zero - tile0;
        if (count <= 0)
            return false;   // only the unit's first places: its tiles are the next CTA's
        unit = Unit(p, entry, u_in, S::kRows);
        now.list = listed ? p.a.indices + ((long long)entry * p.a.queries + unit.query) * p.a.k : nullptr;
        now.row_table =
            p.c.table + ((unsigned)seq < (unsigned)p.c.max_seqs ? seq * p.c.table_stride : 0);
        now.head_pool = p.c.pool + (long long)unit.head * p.c.page_size * S::kRecord;
        now.seen = listed ? len - p.a.queries + 1 + unit.query : len;
        // the warp's tiles: warp, warp + kWarps, ... of `count`
        mine = count > warp && !lost ? (int)((count - warp + S::kWarps - 1) / S::kWarps) : 0;
        // tokens and list entries are below 2^31; the last tile may end above
        e0 = (unsigned)((tile0 + warp) * S::kTile);
        fill = use = 0;
        if constexpr (kRun > 0) {
            run_page = run_page_of(now, 0);
            queries.load(p, unit);
            next_runs(now, 0);
#pragma unroll
            for (int s = 0; s < S::kEarly; ++s)
                if (s < mine)
                    issue_runs(now, s);
        } else {
#pragma unroll
            for (int s = 0; s < S::kStages; ++s)
                early_pos[s] = position(now, s);
#pragma unroll
            for (int s = 0; s < S::kStages; ++s)
                early_page[s] = page_of(now, early_pos[s]);
            queries.load(p, unit);
#pragma unroll
            for (int s = 0; s < S::kEarly; ++s)
                if (s < mine)
                    issue_tokens(now, early_pos[s], early_page[s]);
            pos_after = position(now, S::kStages);
        }
        return true;
    };
    // The unit's query operands and its `Part`, where the last unit's are not
    // needed any more.
    auto announce = [&](int i) {
        queries.store(p, unit, len, smem);
        if (threadIdx.x != 0)
            return;
        volatile Part &part = part_of(i);
        const bool last = u_in + 1 == p.units;
        part.list = now.list, part.row_table = now.row_table;
        part.head_pool = now.head_pool, part.seen = now.seen;
        part.next = zero + tiles;
        part.next_entry = entry + last;
        part.next_unit = last ? 0 : u_in + 1;
        part.active = count < S::kWarps ? (int)count : S::kWarps;
        part.u.b = unit.b, part.u.head = unit.head, part.u.query = unit.query;
        part.u.row0 = unit.row0, part.u.rows = unit.rows;
        part.whole = count == tiles;
        part.begins = tile0 == 0;
        if (tile0 == 0 && count < tiles && !clustered) {
            split->b = entry;
            split->unit = u_in;
            split->parts = (int)(divided(zero + tiles - 1, per) - blockIdx.x) + 1;
        }
    };

    bool more = set_up();
    if (!more)
        return;
    announce(slot);
    __syncthreads();

    while (true) {
        // query operands and `part` are there, the last unit's results are read:
        // the ring's tail can be filled too
        volatile Part &part = part_of(slot);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
#pragma unroll
        for (int s = S::kEarly; s < S::kStages - 1; ++s)
            if (s < mine) {
                if constexpr (kRun > 0)
                    issue_runs(part, s);
                else
                    issue_tokens(part, early_pos[s], early_page[s]);
            }
        if constexpr (kRun == 0)
            pos_next = early_pos[S::kStages - 1], page_next = early_page[S::kStages - 1];

        // Output, and the state of the unit's two rows that this lane shares
        float o[S::kGroups][S::kSubs][4];
        float top[2], sum[2], fac[2];
        float low[2];     // maximum in base-2 units, 0 while there is none
        auto row = [&](int c) { return S::kWide ? g + 8 * c : 2 * t + c; };
        int least = 0x7fffffff;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            top[c] = -INFINITY;
            sum[c] = low[c] = 0.f;
            fac[c] = factor[row(c)];
            if (row(c) < part.u.rows)
                least = min(least, limit[row(c)]);
        }
        // tiles below the lowest limit of any row need no comparison
        least = __reduce_min_sync(~0u, least);
#pragma unroll
        for (int i = 0; i < S::kGroups; ++i)
#pragma unroll
            for (int s = 0; s < S::kSubs; ++s)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    o[i][s][e] = 0.f;
        if (lane < S::kGroups / 2) {
            reinterpret_cast<uint32_t *>(bounds)[lane] = 0;
            reinterpret_cast<uint32_t *>(lifts)[lane] = 0x78007800;     // as of the smallest scale
        }

        // largest of the lanes that share a row
        auto row_max = [&](float v) {
#pragma unroll
            for (int step = S::kWide ? 1 : 4; step < (S::kWide ? 4 : 32); step *= 2)
                v = fmaxf(v, __shfl_xor_sync(~0u, v, step));
            return v;
        };
        // state of accumulator register e: columns 2 t, 2 t + 1 of rows g, g + 8
        auto state = [](int e) { return S::kWide ? e / 2 : e & 1; };
        // Whether a value scale of this lane's token is beyond what the lifts are good
        // for.
        auto beyond = [&](const uint32_t (&w)[S::kGroups / 2]) {
            uint32_t b[S::kGroups / 2];
            load_words(b, bounds);
            bool fits = true;       // a NaN fits any lift
#pragma unroll
            for (int i = 0; i < S::kGroups / 2; ++i)
                fits = fits && __hbleu2(*reinterpret_cast<const __half2 *>(&w[i]),
                                        *reinterpret_cast<const __half2 *>(&b[i]));
            return !fits;
        };
        // New lifts for value scales w of the lanes' tokens, those that count, and the
        // output brought down to them.
        auto lower = [&](const uint32_t (&w)[S::kGroups / 2], bool in) {
            uint32_t b[S::kGroups / 2], bound[S::kGroups / 2] = {}, lift[S::kGroups / 2] = {};
            unsigned most[S::kGroups];
            load_words(b, bounds);
            // (no lift is made for a NaN)
#pragma unroll
            for (int i = 0; i < S::kGroups; ++i) {
                const unsigned s = w[i / 2] >> (i % 2 * 16) & 0xffffu;
                most[i] = __reduce_max_sync(~0u, in && s <= 0x7bffu ? s : 0u);
            }
            auto bits = [](unsigned h) {
                return __float_as_uint(__half2float(__ushort_as_half((unsigned short)h)));
            };
#pragma unroll
            for (int i = 0; i < S::kGroups; ++i) {
                const unsigned old = max(b[i / 2] >> (i % 2 * 16) & 0xffffu, 1u), now = max(most[i], old);
                const float down = __uint_as_float((127u + (bits(old) >> 23) - (bits(now) >> 23)) << 23);
#pragma unroll
                for (int k = 0; k < S::kSubs; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][k][e] *= down;
                // good for every scale of the same exponent
                const unsigned same = now < 0x400u ? (1u << (31 - __clz(now))) - 1 : 0x3ffu;
                bound[i / 2] |= (now | same) << (i % 2 * 16);
                lift[i / 2] |= lift_of(bits(now)) << (i % 2 * 16);
            }
            __syncwarp();       // every lane has read the bounds
            if (lane == 0) {
                store_words(bounds, bound);
                store_words(lifts, lift);
            }
            __syncwarp();
        };
        // New maxima `best` of the lane's scores, or a value scale beyond the lifts.
        // Either is rare after the first tiles: only then the rows' maxima are joined
        // and the sums brought down.  (Looking for the latter and lifting costs 64 x
        // 32768 tokens 403 -> 421 us.)
        auto raise = [&](const float (&best)[2], bool grow, const uint32_t (&w)[S::kGroups / 2], bool in) {
            if (!__any_sync(~0u, best[0] > top[0] || best[1] > top[1] || grow))
                return;
            if (__any_sync(~0u, grow))
                lower(w, in);
            float down[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float m = row_max(fmaxf(best[c], top[c]));
                down[c] = top[c] == -INFINITY ? 0.f : exp2_fast((top[c] - m) * fac[c]);
                top[c] = m;
                low[c] = m == -INFINITY ? 0.f : m * fac[c];
                sum[c] *= down[c];
            }
#pragma unroll
            for (int i = 0; i < S::kGroups; ++i)
#pragma unroll
                for (int s = 0; s < S::kSubs; ++s)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        o[i][s][e] *= down[state(e)];
        };
        // operands of the four codes of each of two tokens in z: codes j of both
        auto value_codes = [](uint32_t z, int j) {
            return j == 0 ? low_codes(z) : j == 1 ? high_codes(z) : j == 2 ? low_codes(z >> 8)
                                                                          : high_codes(z >> 8);
        };

        auto consume = [&](auto masked_tag, const unsigned char *tile, unsigned mask, int base) {
            constexpr bool kMasked = decltype(masked_tag)::value;
            // which of the lane's (token, row) pairs count, a bit each
            unsigned keep = 0;
            auto token_of = [&](int m, int half, int e) {
                return m * 16 + half * S::kNext + (!S::kWide ? tok_row : e & 1 ? tok_b : tok_a);
            };
            if constexpr (kMasked) {
                const int seen[2] = {listed ? 0x7fffffff : limit[row(0)] - base,
                                     listed ? 0x7fffffff : limit[row(1)] - base};
#pragma unroll
                for (int m = 0; m < S::kMT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int e = 0; e < (S::kWide ? 4 : 2); ++e) {
                            const int token = token_of(m, half, e), c = S::kWide ? e / 2 : e;
                            if ((mask >> token & 1) && token < seen[c])
                                keep |= 1u << ((m * 2 + half) * 4 + e);
                        }
            }
            auto kept = [&](int m, int half, int e) { return keep >> ((m * 2 + half) * 4 + e) & 1; };
            // a token each for the lanes: its value scales (the last row sees most tokens)
            const int token = lane % S::kTile;
            const bool in = !kMasked || ((mask >> token & 1) &&
                                         (listed || base + token < limit[part.u.rows - 1]));
            uint32_t scales[S::kGroups / 2], lift[S::kGroups / 2];
            load_words(scales, tile + token * S::kRecord + D + 2 * S::kGroups);
            const bool grow = in && beyond(scales);
            if constexpr (!S::kWide) {
                float sc[S::kMT][4], sa[S::kMT][S::kGroups], sb[S::kMT][S::kGroups];
#pragma unroll
                for (int mt = 0; mt < S::kMT; ++mt) {
                    const unsigned char *ra = tile + (mt * 16 + tok_row) * S::kRecord;
                    load_scales(sa[mt], ra + D);
                    load_scales(sb[mt], ra + S::kNext * S::kRecord + D);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sc[mt][e] = 0.f;
                }
#pragma unroll
                for (int st = 0; st < S::kStretches; ++st) {
                    uint32_t wa[S::kMT][S::kPer], wb[S::kMT][S::kPer];
#pragma unroll
                    for (int mt = 0; mt < S::kMT; ++mt) {
                        const unsigned char *ra =
                            tile + (mt * 16 + tok_row) * S::kRecord + st * 64 + t * S::kPer * 4;
                        load_words(wa[mt], ra);
                        load_words(wb[mt], ra + S::kNext * S::kRecord);
                    }
#pragma unroll
                    for (int i = 0; i < S::kPer; ++i) {
                        const int group = st * S::kPer + i;
                        const uint2 *qf = reinterpret_cast<const uint2 *>(smem + S::kOffQ) + group * 2 * 32 + lane;
                        const uint2 q0 = qf[0], q1 = qf[32];
#pragma unroll
                        for (int mt = 0; mt < S::kMT; ++mt) {
                            const uint32_t la = wa[mt][i], lb = wb[mt][i], ha = la >> 8, hb = lb >> 8;
                            float acc[4] = {0.f, 0.f, 0.f, 0.f};
                            mma16816(acc, low_codes(la), low_codes(lb), high_codes(la), high_codes(lb), q0.x,
                                     q0.y);
                            mma16816(acc, low_codes(ha), low_codes(hb), high_codes(ha), high_codes(hb), q1.x,
                                     q1.y);
                            sc[mt][0] += sa[mt][group] * acc[0];
                            sc[mt][1] += sa[mt][group] * acc[1];
                            sc[mt][2] += sb[mt][group] * acc[2];
                            sc[mt][3] += sb[mt][group] * acc[3];
                        }
                    }
                }
                float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int mt = 0; mt < S::kMT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kMasked && !kept(mt, e / 2, e & 1))
                            sc[mt][e] = -INFINITY;
                        best[e & 1] = fmaxf(best[e & 1], sc[mt][e]);
                    }
                raise(best, grow, scales, in);
                load_words(lift, lifts);
                // (masked tiles are rare: their code is kept short, which the other
                // tiles gain 2 % from)
#pragma unroll (kMasked ? 1 : S::kMT)
                for (int mt = 0; mt < S::kMT; ++mt) {
                    const unsigned char *ra = tile + (mt * 16 + tok_row) * S::kRecord;
                    float sa[S::kGroups], sb[S::kGroups], pr[4];
                    load_lifted(sa, ra + D + 2 * S::kGroups, lift);
                    load_lifted(sb, ra + S::kNext * S::kRecord + D + 2 * S::kGroups, lift);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        pr[e] = exp2_fast(sc[mt][e] * fac[e & 1] - low[e & 1]);
                        if (kMasked && !kept(mt, e / 2, e & 1))
                            pr[e] = 0.f;
                        sum[e & 1] += pr[e];
                        pr[e] *= kRaise;
                    }
                    const unsigned char *va = tile + (mt * 16 + tok_a) * S::kRecord + D / 2;
                    const unsigned char *vb = tile + (mt * 16 + tok_b) * S::kRecord + D / 2;
#pragma unroll
                    for (int st = 0; st < S::kStretches; ++st) {
                        constexpr int kW = S::kPer / 2;
                        uint32_t wa[kW], wb[kW], xa[kW], xb[kW];
                        load_words(wa, va + st * 64 + g * kW * 4);
                        load_words(wb, vb + st * 64 + g * kW * 4);
                        load_words(xa, va + S::kNext * S::kRecord + st * 64 + g * kW * 4);
                        load_words(xb, vb + S::kNext * S::kRecord + st * 64 + g * kW * 4);
#pragma unroll
                        for (int i = 0; i < S::kPer; ++i) {
                            const int group = st * S::kPer + i;
                            const uint32_t z = __byte_perm(wa[i / 2], wb[i / 2], i & 1 ? 0x7632 : 0x5410);
                            const uint32_t y = __byte_perm(xa[i / 2], xb[i / 2], i & 1 ? 0x7632 : 0x5410);
                            float w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                w[e] = pr[e] * (e < 2 ? sa[group] : sb[group]);
                                // whatever the record holds
                                if (kMasked && !kept(mt, e / 2, e & 1))
                                    w[e] = 0.f;
                            }
                            const uint32_t b0 = transpose8x8(pack_half2(w[0], w[1]));
                            const uint32_t b1 = transpose8x8(pack_half2(w[2], w[3]));
                            mma16816(o[group][0], value_codes(z, 0), value_codes(z, 1),
                                     value_codes(y, 0), value_codes(y, 1), b0, b1);
                            mma16816(o[group][1], value_codes(z, 2), value_codes(z, 3),
                                     value_codes(y, 2), value_codes(y, 3), b0, b1);
                        }
                    }
                }
            } else {
                // scores of a step's places 2 t, 2 t + 1 (half 0) and those + 8
                float sc[S::kMT][2][4];
                const int next = S::kNext * S::kRecord;
                auto record = [&](int m, int token) {
                    return tile + (m * 16 + token) * S::kRecord;
                };
#pragma unroll
                for (int m = 0; m < S::kMT; ++m) {
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const unsigned char *rk = record(m, tok_row) + half * next;
                        float sa[S::kGroups], sb[S::kGroups];
                        load_scales(sa, record(m, tok_a) + half * next + D);
                        load_scales(sb, record(m, tok_b) + half * next + D);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            sc[m][half][e] = 0.f;
#pragma unroll
                        for (int st = 0; st < S::kStretches; ++st) {
                            uint32_t wk[S::kPer];
                            load_words(wk, rk + st * 64 + t * S::kPer * 4);
#pragma unroll
                            for (int i = 0; i < S::kPer; ++i) {
                                const int group = st * S::kPer + i;
                                const uint32_t k0 = low_codes(wk[i]), k1 = high_codes(wk[i]);
                                const uint32_t k2 = low_codes(wk[i] >> 8), k3 = high_codes(wk[i] >> 8);
                                const uint4 *qf = reinterpret_cast<const uint4 *>(smem + S::kOffQ) +
                                                  group * 2 * 32 + lane;
                                const uint4 q0 = qf[0], q1 = qf[32];
                                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                                mma16816(acc, q0.x, q0.y, q0.z, q0.w, k0, k1);
                                mma16816(acc, q1.x, q1.y, q1.z, q1.w, k2, k3);
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    sc[m][half][e] += (e & 1 ? sb[group] : sa[group]) * acc[e];
                            }
                        }
                    }
                }
                float best[2];
                best[0] = best[1] = -INFINITY;
#pragma unroll
                for (int m = 0; m < S::kMT; ++m)
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            if (kMasked && !kept(m, half, e))
                                sc[m][half][e] = -INFINITY;
                            best[e / 2] = fmaxf(best[e / 2], sc[m][half][e]);
                        }
                raise(best, grow, scales, in);
                load_words(lift, lifts);
#pragma unroll
                for (int m = 0; m < S::kMT; ++m) {
#pragma unroll
                    for (int half = 0; half < 2; ++half)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float pr = exp2_fast(sc[m][half][e] * fac[e / 2] - low[e / 2]);
                            if (kMasked && !kept(m, half, e))
                                pr = 0.f;
                            sum[e / 2] += pr;
                            sc[m][half][e] = pr * kRaise;
                        }
                    const unsigned char *ra = record(m, tok_a), *rb = record(m, tok_b);
                    float vs[4][S::kGroups];     // value scales of the lane's four tokens
                    load_lifted(vs[0], ra + D + 2 * S::kGroups, lift);
                    load_lifted(vs[1], rb + D + 2 * S::kGroups, lift);
                    load_lifted(vs[2], ra + next + D + 2 * S::kGroups, lift);
                    load_lifted(vs[3], rb + next + D + 2 * S::kGroups, lift);
#pragma unroll
                    for (int st = 0; st < S::kStretches; ++st) {
                        constexpr int kW = S::kPer / 2;
                        const int at = D / 2 + st * 64 + g * kW * 4;
                        uint32_t wa[kW], wb[kW], xa[kW], xb[kW];
                        load_words(wa, ra + at);
                        load_words(wb, rb + at);
                        load_words(xa, ra + next + at);
                        load_words(xb, rb + next + at);
#pragma unroll
                        for (int i = 0; i < S::kPer; ++i) {
                            const int group = st * S::kPer + i;
                            const uint32_t z = __byte_perm(wa[i / 2], wb[i / 2], i & 1 ? 0x7632 : 0x5410);
                            const uint32_t y = __byte_perm(xa[i / 2], xb[i / 2], i & 1 ? 0x7632 : 0x5410);
                            uint32_t pa[4];
                            float w[2][4];
#pragma unroll
                            for (int half = 0; half < 2; ++half)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    w[half][e] = sc[m][half][e] * vs[half * 2 + (e & 1)][group];
                                    if (kMasked && !kept(m, half, e))
                                        w[half][e] = 0.f;
                                }
                            pa[0] = pack_half2(w[0][0], w[0][1]);
                            pa[1] = pack_half2(w[0][2], w[0][3]);
                            pa[2] = pack_half2(w[1][0], w[1][1]);
                            pa[3] = pack_half2(w[1][2], w[1][3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t b0 = value_codes(z, j), b1 = value_codes(y, j);
                                mma16816(o[group][j], pa[0], pa[1], pa[2], pa[3], b0, b1);
                            }
                        }
                    }
                }
            }
        };

        for (int i = 0; i < mine; ++i) {
            // every lane is done with the stage that is filled next
            __syncwarp();
            if constexpr (kRun > 0) {
                if (i + S::kStages - 1 < mine)
                    issue_runs(part, i + S::kStages - 1);
            } else {
                if (i + S::kStages - 1 < mine)
                    issue_tokens(part, pos_next, page_next);
                pos_next = pos_after;
                page_next = page_of(part, pos_next);
                pos_after = position(part, i + S::kStages + 1);
            }

            const unsigned mask = masks[use];
            barrier_wait(barriers + use * 8, phases >> use & 1, late);
            phases ^= 1u << use;
            const unsigned char *data = ring + use * S::kStageBytes;
            use = use + 1 == S::kStages ? 0 : use + 1;
            const int base = listed ? 0 : (int)(e0 + i * (S::kWarps * S::kTile));
            if (mask == S::kFullMask && (listed || base + S::kTile <= least))
                consume(std::false_type{}, data, mask, base);
            else if (mask)
                consume(std::true_type{}, data, mask, base);
        }
        // What came too late was taken as it was, by all lanes alike; now they agree
        // that it was lost, and give what is still under way as long again.
        if (__any_sync(~0u, late)) {
            lost = true;
            late = false;
            for (int s = 0; s < S::kStages; ++s)
                barrier_wait(barriers + s * 8, ~phases >> s & 1, late);
            __syncwarp();
        }

        const int active = part.active;
        // ---- the warps' results in their rings' tails (a warp without tiles
        // has none) ----------------------------------------------------------
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (warp >= active)
                break;
            const int r = row(c);
            float s = lost ? __int_as_float(0x7fffffff) : sum[c];
#pragma unroll
            for (int step = S::kWide ? 1 : 4; step < (S::kWide ? 4 : 32); step *= 2)
                s += __shfl_xor_sync(~0u, s, step);
            if (S::kWide ? t == 0 : g == 0) {
                wmax(warp, r) = top[c] == -INFINITY ? -INFINITY : low[c];
                wsum(warp, r) = s;
            }
            // narrow: rows of the instruction are channels 4 g + {0, 1} and
            // 4 g + {2, 3}; wide: columns 2 t, 2 t + 1 of instruction j are
            // channels 8 t + j and 8 t + 4 + j.  Odd ones are 16 times too large, and
            // all of a group by its lift.
            float *dst = reinterpret_cast<float *>(ring + S::kTail) + r * S::kOutStride;
#pragma unroll
            for (int i = 0; i < S::kGroups; ++i) {
                const float back = lift_back(reinterpret_cast<const unsigned short *>(lifts)[i]);
                const float back16 = back * 0.0625f;
                if constexpr (S::kWide) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        *reinterpret_cast<float4 *>(dst + i * kGroup + 8 * t + 4 * k) = make_float4(
                            o[i][0][2 * c + k] * back, o[i][1][2 * c + k] * back16,
                            o[i][2][2 * c + k] * back, o[i][3][2 * c + k] * back16);
                } else {
                    *reinterpret_cast<float4 *>(dst + i * kGroup + 4 * g) =
                        make_float4(o[i][0][c] * back, o[i][0][c + 2] * back16, o[i][1][c] * back,
                                    o[i][1][c + 2] * back16);
                }
            }
        }

        // ---- the unit after this one, under way while the results are joined -
        x = start = clustered ? end : part.next;
        entry = part.next_entry;
        u_in = part.next_unit;
        more = set_up();
        __syncthreads();
        if (more)
            announce(slot ^ 1);

        Unit u;
        u.b = part.u.b, u.head = part.u.head, u.query = part.u.query;
        u.row0 = part.u.row0, u.rows = part.u.rows;
        const bool whole = part.whole;
        // a CTA's second place is for the unit that begins in it
        float *to_join = p.a.partial + p.parts + (blockIdx.x * 2LL + part.begins) * S::kPartial;
        // Four channels of a row: maximum, sum and output of all parts i < n, which
        // weigh 2^(maximum - largest maximum).  A part that saw nothing has maximum
        // -inf and sum 0; one whose scores are NaN has maximum -inf, and its NaN
        // goes on.
        struct Four {
            float m, l;
            float4 v;
        };
        auto add_up = [&](auto most, int n, auto maximum, auto sum_of, auto output) {
            constexpr int kMost = decltype(most)::value;      // n is at most this
            Four f = {-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
            float m[kMost];
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                m[i] = i < n ? maximum(i) : -INFINITY;
                f.m = fmaxf(f.m, m[i]);
            }
#pragma unroll
            for (int i = 0; i < kMost; ++i) {
                if (i >= n)
                    break;
                const float s = sum_of(i);
                const float weight = s == 0.f ? 0.f : s != s ? 1.f : exp2_fast(m[i] - f.m);
                const float4 o4 = output(i);
                f.l += s * weight;
                f.v.x += o4.x * weight, f.v.y += o4.y * weight;
                f.v.z += o4.z * weight, f.v.w += o4.w * weight;
            }
            return f;
        };
        auto of_warps = [&](int r, int d) {
            return add_up(std::integral_constant<int, S::kWarps>(), active, [&](int w) { return wmax(w, r); },
                          [&](int w) { return wsum(w, r); },
                          [&](int w) {
                              return *reinterpret_cast<const float4 *>(
                                  smem + w * S::kWarpBytes + S::kTail + (r * S::kOutStride + d) * 4);
                          });
        };
        auto finish = [&](int r, int d, const Four &f) {
            int j, h;
            u.row(p, r, &j, &h);
            const long long at = ((long long)u.b * p.a.queries + j) * p.a.heads + h;
            const float inv = f.l == 0.f ? 0.f : 1.f / f.l;
            if (p.a.bf16)
                store_four((__nv_bfloat16 *)p.a.out + at * D + d, f.v, inv);
            else
                store_four((__half *)p.a.out + at * D + d, f.v, inv);
            if (d == 0 && p.a.lse)
                p.a.lse[at] = f.l == 0.f ? -INFINITY : (f.m + log2f(f.l)) * 0.6931471805599453f;
        };
        constexpr int kFours = S::kRows * D / 4;
        if constexpr (kRun == 0) {
            if (clustered) {
                // this CTA's part into its shared memory, then every CTA of the
                // cluster joins its share of the rows from all of them
                constexpr int kMine = (kFours + S::kThreads - 1) / S::kThreads;
                Four f[kMine];
#pragma unroll
                for (int n = 0; n < kMine; ++n) {
                    const int e = threadIdx.x + n * S::kThreads, r = e / (D / 4);
                    if (r < u.rows)
                        f[n] = of_warps(r, e % (D / 4) * 4);
                }
                __syncthreads();
                float *mine = reinterpret_cast<float *>(smem);     // maxima, sums, outputs
#pragma unroll
                for (int n = 0; n < kMine; ++n) {
                    const int e = threadIdx.x + n * S::kThreads, r = e / (D / 4), d = e % (D / 4) * 4;
                    if (r < u.rows) {
                        *reinterpret_cast<float4 *>(mine + 2 * S::kRows + r * D + d) = f[n].v;
                        if (d == 0)
                            mine[r] = f[n].m, mine[S::kRows + r] = f[n].l;
                    }
                }
                cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
                cluster.sync();
                for (int e = threadIdx.x + cluster.block_rank() * S::kThreads; e < kFours;
                     e += p.cluster * S::kThreads) {
                    const int r = e / (D / 4), d = e % (D / 4) * 4;
                    if (r >= u.rows)
                        break;
                    auto of = [&](int i) { return cluster.map_shared_rank(mine, i); };
                    finish(r, d, add_up(std::integral_constant<int, 8>(), p.cluster,
                                        [&](int i) { return of(i)[r]; },
                                        [&](int i) { return of(i)[S::kRows + r]; },
                                        [&](int i) {
                                            return *reinterpret_cast<const float4 *>(
                                                of(i) + 2 * S::kRows + r * D + d);
                                        }));
                }
                cluster.sync();     // the others have read this CTA's part
                return;
            }
        }
        for (int e = threadIdx.x; e < kFours; e += S::kThreads) {
            const int r = e / (D / 4), d = e % (D / 4) * 4;
            if (r >= u.rows)
                break;
            const Four f = of_warps(r, d);
            if (whole) {
                finish(r, d, f);
            } else {
                *reinterpret_cast<float4 *>(to_join + 2 * S::kRows + r * D + d) = f.v;
                if (d == 0) {
                    to_join[r] = f.m;
                    to_join[S::kRows + r] = f.l;
                }
            }
        }
        if (!more)
            break;
        __syncthreads();
        slot ^= 1;
    }
}

// Joins the partial results of units that several CTAs worked on: for the unit
// that began in attending CTA blockIdx.x / (Rows / 8), a warp a query row, parts
// in order.  All CTAs together have at most two parts each, so that many parts
// of one unit mean few units.
constexpr int kJoinThreads = 256;

template <int D, int Rows>
__global__ void __launch_bounds__(kJoinThreads)
join_kernel(const __grid_constant__ AttendArgs p)
{
    using S = Shape<D, Rows>;
    constexpr int kMine = D / 32, kAhead = 32 / kMine;      // channels of a lane; parts under way
    const int lane = threadIdx.x & 31;
    const int cta = blockIdx.x / (Rows / 8), r = blockIdx.x % (Rows / 8) * 8 + threadIdx.x / 32;
    dependent_grid_wait();
    allow_dependent_grid();
    const int4 split = reinterpret_cast<const int4 *>(p.a.partial)[cta];
    const int parts = split.z;
    if (parts == 0)
        return;
    const Unit u(p, split.x, split.y, Rows);
    if (r >= u.rows)
        return;
    // a CTA's second place holds the unit that begins in it
    const float *base = p.a.partial + p.parts + 2LL * cta * S::kPartial;
    auto place = [&](int i) { return base + (i == 0 ? 1 : 2 * i) * (long long)S::kPartial; };
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32)
        m = fmaxf(m, place(i)[r]);
#pragma unroll
    for (int step = 16; step; step /= 2)
        m = fmaxf(m, __shfl_xor_sync(~0u, m, step));
    const float low = m == -INFINITY ? 0.f : m;
    float l = 0.f, v[kMine];
#pragma unroll
    for (int c = 0; c < kMine; ++c)
        v[c] = 0.f;
    for (int i0 = 0; i0 < parts; i0 += kAhead) {
        float f[kAhead][kMine], weight[kAhead], s[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const bool in = i0 + k < parts;
            const float *q = place(in ? i0 + k : 0);
            s[k] = in ? q[S::kRows + r] : 0.f;
            weight[k] = in ? q[r] : -INFINITY;
#pragma unroll
            for (int c = 0; c < kMine; ++c)
                f[k][c] = in ? q[2 * S::kRows + r * D + c * 32 + lane] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const float w = s[k] != s[k] ? 1.f : exp2_fast(weight[k] - low);
            l += s[k] * w;
#pragma unroll
            for (int c = 0; c < kMine; ++c)
                v[c] += f[k][c] * w;
        }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    int j, h;
    u.row(p, r, &j, &h);
    const long long row = ((long long)u.b * p.a.queries + j) * p.a.heads + h;
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
        if (p.a.bf16)
            from_float(((__nv_bfloat16 *)p.a.out)[row * D + c * 32 + lane], v[c] * inv);
        else
            from_float(((__half *)p.a.out)[row * D + c * 32 + lane], v[c] * inv);
    }
    if (p.a.lse && lane == 0)
        p.a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// ---- host ----------------------------------------------------------------------
// Query rows of a unit: 8, or 16 where there are more.  Further rows are further
// units.  Units of 32 rows would expand a record once instead of twice, but their
// outputs leave 8 warps an SM that cannot hide each other's waits (32 rows, 16 x
// 16384 tokens: 197 us in one unit where two took 186, which take 180 now; 80
// rows, 4 x 65536: 94 and 72, now 70).
inline int unit_rows(int rows) { return rows <= 8 ? 8 : 16; }

// How a call is laid out: sizes of its units, its CTAs, and whether units are
// cut between CTAs.  They are not, and the join is saved, where a unit is at
// most two tiles a warp, and where tokens are listed, so that all units are of
// one known size, and whole ones keep at least half of one wave of CTAs or four
// fifths of several busy (512 of 32768 tokens, 128 units for 152 CTAs: 20.5
// instead of 28.7 us; 64 units of 2048 tokens for 304 CTAs: 24.6 cut, 30.7 whole).
// Between one wave and four fifths of two they are cut (1024 tokens: 320 units 38.9
// us cut, 45.1 whole in persistent CTAs, 41.0 whole in a CTA each; 384 units 43.0,
// 45.1, 41.0; 440 units 47.1, 45.1, 47.1).
template <int D, int Rows>
int lay_out(AttendArgs &p, int sms)
{
    using S = Shape<D, Rows>;
    p.blocks = (p.rows + S::kRows - 1) / S::kRows;
    p.units = p.c.kv_heads * p.blocks * (p.a.k > 0 ? p.a.queries : 1);
    p.sel_tiles = ((long long)p.a.k + S::kTile - 1) / S::kTile;
    const double room = (double)p.c.max_pages * p.c.page_size;
    const double tiles = p.a.k > 0 ? (double)p.sel_tiles : room / S::kTile + 1;   // of a unit, at most
    const double units = (double)p.units * p.a.batch, ctas = (double)sms * S::kCtas;
    const double waves = (double)(long long)((units + ctas - 1) / ctas);
    p.whole = tiles <= 2 * S::kWarps ||
              (p.a.k > 0 && units >= (units <= ctas ? 0.5 * ctas : 0.8 * ctas * waves));
    // Few listed units of middling size: a cluster of CTAs each, which joins its
    // parts in shared memory, while that gives no warp more than four tiles
    // (64 units of 2048 tokens, four CTAs each: 20.5 us, with a join launch 24.6).
    p.cluster = 1;
    if (p.a.k > 0 && !p.whole) {
        while (p.cluster < 8 && tiles > 2 * S::kWarps * p.cluster && 2 * p.cluster * units <= ctas)
            p.cluster *= 2;
        if (p.cluster > 1 && tiles <= 4 * S::kWarps * p.cluster)
            return (int)(units * p.cluster);
        p.cluster = 1;
    }
    // no more CTAs than the largest possible line has work for
    const double most = p.whole ? units : (tiles + kUnitCost) * units / (2 * S::kWarps) + 1;
    return (int)(most < ctas ? most : ctas);
}

template <int D, int Rows>
cudaError_t launch_shape(AttendArgs &p, int dev, int sms, cudaStream_t stream)
{
    using S = Shape<D, Rows>;
    const int ctas = lay_out<D, Rows>(p, sms);
    p.by_group.set(p.group);
    p.by_blocks.set(p.blocks);
    p.by_heads.set(p.c.kv_heads);
    p.parts = ctas * (long long)(sizeof(Split) / sizeof(float));
    const int which = p.a.k > 0 || p.run < 16 ? 0 : p.run == S::kTile ? 1 : 2;
    auto fn = which == 0   ? attend_kernel<D, Rows, 0>
              : which == 1 ? attend_kernel<D, Rows, S::kTile> : attend_kernel<D, Rows, 16>;
    // the kernels' shared memory is raised once a device
    static std::atomic<unsigned long long> raised[3];
    cudaError_t e = cudaSuccess;
    if (!(raised[which].load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess)
            return e;
        raised[which].fetch_or(1ULL << dev, std::memory_order_relaxed);
    }
    e = launch_clusters(fn, p.cluster, ctas, S::kThreads, S::kSmem, stream, p);
    if (e != cudaSuccess || p.whole || p.cluster > 1)
        return e;
    return launch_overlapped(join_kernel<D, Rows>, ctas * (Rows / 8), kJoinThreads, 0, stream, p);
}

// The arguments that the layout goes by.
template <int D>
AttendArgs attend_args(const Cache &c, const Attend &a)
{
    AttendArgs p;
    p.c = c;
    p.a = a;
    p.group = a.heads / c.kv_heads;
    p.rows = a.k > 0 ? p.group : p.group * a.queries;
    p.run = 1;
    while (a.k == 0 && p.run < Shape<D, 8>::kTile && c.page_size % (2 * p.run) == 0)
        p.run *= 2;
    return p;
}

template <int D>
cudaError_t launch_dim(const Cache &c, const Attend &a, int dev, int sms, cudaStream_t stream)
{
    AttendArgs p = attend_args<D>(c, a);
    return unit_rows(p.rows) == 8 ? launch_shape<D, 8>(p, dev, sms, stream)
                                  : launch_shape<D, 16>(p, dev, sms, stream);
}

template <int D, int Rows>
size_t workspace_shape(AttendArgs &p, int sms)
{
    const int ctas = lay_out<D, Rows>(p, sms);
    return p.whole || p.cluster > 1 ? 0 : ctas * (sizeof(Split) + 2 * Shape<D, Rows>::kPartial * sizeof(float));
}

template <int D>
size_t workspace_dim(const Cache &c, const Attend &a, int sms)
{
    AttendArgs p = attend_args<D>(c, a);
    return unit_rows(p.rows) == 8 ? workspace_shape<D, 8>(p, sms) : workspace_shape<D, 16>(p, sms);
}

}  // namespace kv4
}  // namespace ds
