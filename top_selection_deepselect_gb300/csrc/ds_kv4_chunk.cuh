// ds_kv4_chunk.cuh -- attention of chunks of new tokens over the 4-bit cache.
//
// A chunk has many query rows for each key/value head, so that the products
// bound it and not the records: S = Q K^T and O = P V go to the fifth-generation
// tensor cores, 128 rows and 64 tokens at a time, with Q, S, P and O in tensor
// memory and the expanded keys and values in shared memory.
//
// Rows.  The (query, head) pairs of a key/value head's group, head fastest, are
// the rows of one problem; a unit is a block of up to kTiles x 128 of them.  With
// two tiles of rows the tensor cores work on one while the other's softmax is
// taken; a tile of tokens is expanded once for both.
//
// Exact scores.  A key's channel is (u - 8) scale, three bits times eleven, which
// does not fit a 16-bit operand.  The scale is split into two numbers of few
// enough bits that both products are exact, and S is the sum of Q times each:
// half as many operations more, and log-sums as exact as 32-bit arithmetic has
// them.  Queries stay as they are: the operands' type is theirs.  Probabilities and
// values are fp16 in the second product, whatever the queries' type, each rounded
// to 11 bits once; powers of two keep both within its range.
//
// Codes become operands by a logical operation and a packed multiply-add or addition:
// a code u in the low bits of an fp16 of 1024 makes it 1024 + u, and subtracting 1032
// leaves u - 8; in the upper bits of the fraction of a bf16 of 16 it makes 16 + u, and
// (16 + u) s - 24 s is exact for a part s of a scale.  A word of eight key codes gives
// channels (j, j + 4) in pairs; the queries are laid out in the same order.  A value's
// word is taken with that of the next token, so that pairs are (token, token + 1)
// of one channel: both operands end up with the summed index contiguous.
//
// What bounds it.  For 64 tokens and 256 rows of 128 channels the products take 1536
// cycles of the tensor cores, a third of them for the keys' second part, and the four
// schedulers issue some 1600 instructions each: 330 a tile of rows for weights and
// maxima, 290 for keys, 230 for values, the rest for waits and what surrounds them.
// 2048 tokens of 32768 (64 query heads, 8 key/value heads of 128, bf16) take 1.97 ms:
// 1080 TFLOP/s, 1620 with the second part, which is 84 % of what a large bf16 library
// product reaches in a burst; over many calls in turn the power limit brings it to
// 2.05 to 2.12 ms.  Heads of 64 and 256 stay at 500 and 630 TFLOP/s: there the expansion
// and the softmax are as large for a half of the products, or serve 128 rows (1024 tokens
// after 7168: issue slots 62 and 53 % busy, the tensor pipe 37 and 44 %, else the roles'
// waits for each other).
//
// Roles of a CTA's warps: softmax (eight warps a tile of rows, half a row a thread),
// expansion of keys and of values (four warps each, eight for D = 256), one that issues
// the products, one that copies records.  They meet on arrival barriers in shared
// memory.  (A whole row a thread, with registers shifted between the roles, was 5 %
// slower; 64-bit register pairs for the weights 3 %; rolled loops for less code, in any
// of the roles' inner loops, 5 to 8 %.)
//
// Work is a line of places: every (unit, head) has places for each of its tiles of
// tokens, and for its start and end, by what these take; CTAs, one an SM, have
// equal stretches.  Units cut between CTAs leave partial results for a last launch.
// Lengths and starts are read on the device by a first, small launch, or where there is
// little to do by each CTA.
#pragma once

#include <atomic>
#include <type_traits>

#include "ds_device.cuh"
#include "ds_host.h"
#include "ds_kv4.cuh"
#include "ds_kv4_chunk.h"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {
namespace chunk {

constexpr int kTokens = 64;            // of a tile
constexpr int kTileRows = 128;         // query rows of a product
constexpr float kLog2e = 1.4426950408889634f;

template <int D>
struct Shape {
    static constexpr int kTiles = tiles_of_rows(D);
    static constexpr int kRows = kTiles * kTileRows;
    static constexpr int kRecord = record_bytes(D);
    // Records lie in shared memory in groups of eight tokens, 16 bytes further
    // apart than their size: the eight lanes of a load then meet different banks.
    static constexpr int kGroupBytes = 8 * kRecord + 16;
    static constexpr int kRawBytes = kTokens / 8 * kGroupBytes;
    static constexpr int kKeyBytes = kTokens * D * 2;          // of one part of the split
    static constexpr int kValueBytes = kTokens * D * 2;
    // Stages, as many as there is room for.  Two or four for D <= 128 change nothing
    // (2.00 and 2.02 ms where three took 2.01).  For D = 256 a second stage of values took
    // 461 us in the place of a second of keys, and 488 us in the place of two of records,
    // where one takes 412 (1024 tokens after 7168).
    static constexpr int kKeyStages = D == 256 ? 2 : 3;
    static constexpr int kValueStages = D == 256 ? 1 : 3;
    static constexpr int kRawStages = 3;
    // warps
    static constexpr int kSoftmaxWarps = 8 * kTiles;
    // Of each four warps after them two expand keys and two values: a scheduler (warps
    // of one number modulo 4) then has one of the two roles' instructions to fetch.
    static constexpr int kExpandWarp = kSoftmaxWarps, kExpandWarps = D == 256 ? 16 : 8;
    static constexpr int kExpandThreads = 16 * kExpandWarps;     // for keys, and for values
    static constexpr int kProductWarp = kExpandWarp + kExpandWarps, kCopyWarp = kProductWarp + 1;
    static constexpr int kThreads = 32 * (kCopyWarp + 1);
    // columns of tensor memory
    static constexpr int kOutColumn = 0;
    static constexpr int kScoreColumn = kTiles * D;             // two of them
    static constexpr int kQueryColumn = kScoreColumn + 2 * kTokens;
    static_assert(kQueryColumn + kTiles * D / 2 <= 512, "tensor memory");
    // shared memory, from a 1024-byte boundary
    static constexpr int kOffKeys = 0;
    static constexpr int kOffValues = kOffKeys + kKeyStages * 2 * kKeyBytes;
    static constexpr int kOffRaw = kOffValues + kValueStages * kValueBytes;
    static constexpr int kUsed = kOffRaw + kRawStages * kRawBytes + 1024;
    // tensor memory is taken whole, so that a second CTA would only wait for it
    static constexpr int kSmem = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
    static_assert(kSmem <= 217 * 1024, "shared memory of an SM, less what is not of the stages");
    static constexpr int kPartial = kRows * (D + 2);            // floats of a partial result
};

// ---- barriers ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t shared_at(const void *p)
{
    return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void bar_init(uint32_t bar, unsigned count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, unsigned bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_done(uint32_t bar, unsigned phase)
{
    unsigned done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done) : "r"(bar), "r"(phase) : "memory");
    return done != 0;
}
__device__ __forceinline__ long long clock_ns()
{
    long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Nanoseconds that anything is waited for, far beyond what a working GPU takes.
constexpr long long kPatience = 1000000000;

// Waits for a phase to end.  *lost: a wait was given up, by whichever warp; nothing
// is waited for any more, and results are NaN.
__device__ __forceinline__ void bar_wait(uint32_t bar, unsigned phase, volatile int *lost)
{
    long long from = 0;
    for (unsigned tries = 1; !bar_done(bar, phase); ++tries) {
        if (tries % 8 != 0)
            continue;
        if (*lost)
            return;
        if (tries % 64 != 0)               // the timer takes longer to read than most waits
            continue;
        const long long now = clock_ns();
        if (from == 0)
            from = now;
        if (now - from > kPatience) {
            *lost = 1;
            return;
        }
    }
}

// Turn of a ring of n stages: which stage, and the phase its next use ends.
template <int n>
struct Turn {
    int stage = 0;
    unsigned phase = 0;
    __device__ __forceinline__ void step()
    {
        if (++stage == n)
            stage = 0, phase ^= 1;
    }
};

// ---- tensor memory and products --------------------------------------------------
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void fence_proxy() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 32 columns of the warp's 32 rows, a row a lane.
__device__ __forceinline__ void load_columns(uint32_t (&x)[32], uint32_t at)
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
        "%27,%28,%29,%30,%31}, [%32];"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]),
          "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]),
          "=r"(x[15]), "=r"(x[16]), "=r"(x[17]), "=r"(x[18]), "=r"(x[19]), "=r"(x[20]), "=r"(x[21]),
          "=r"(x[22]), "=r"(x[23]), "=r"(x[24]), "=r"(x[25]), "=r"(x[26]), "=r"(x[27]), "=r"(x[28]),
          "=r"(x[29]), "=r"(x[30]), "=r"(x[31])
        : "r"(at));
}
__device__ __forceinline__ void store_columns(uint32_t at, const uint32_t (&x)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,"
        "%27,%28,%29,%30,%31,%32};" ::"r"(at),
        "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]),
        "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15]), "r"(x[16]),
        "r"(x[17]), "r"(x[18]), "r"(x[19]), "r"(x[20]), "r"(x[21]), "r"(x[22]), "r"(x[23]), "r"(x[24]),
        "r"(x[25]), "r"(x[26]), "r"(x[27]), "r"(x[28]), "r"(x[29]), "r"(x[30]), "r"(x[31])
        : "memory");
}

__device__ __forceinline__ void load_columns(uint32_t (&x)[16], uint32_t at)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]),
                   "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]),
                   "=r"(x[14]), "=r"(x[15])
                 : "r"(at));
}
__device__ __forceinline__ void store_columns(uint32_t at, const uint32_t (&x)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(at),
                 "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]),
                 "r"(x[8]), "r"(x[9]), "r"(x[10]), "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
                 : "memory");
}

// Operand in shared memory: rows of 128 bytes (64 numbers of the summed index),
// eight of them a block of 1024 bytes, 16-byte pieces at place (piece ^ row % 8).
// Its descriptor's lower word; the upper one says the blocks' distance, and the order.
__device__ __forceinline__ uint32_t operand_at(uint32_t at) { return (at >> 4) | 1u << 16; }
constexpr uint32_t kOperandKind = 1024 >> 4 | 1u << 14 | 2u << 29;
// 16-bit operands of one type, 32-bit sums, 128 rows, n columns.
template <typename T>
__device__ __forceinline__ constexpr uint32_t product_of(int n)
{
    constexpr uint32_t type = sizeof(T) == 2 && std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
    return 1u << 4 | type << 7 | type << 10 | (uint32_t)(n >> 3) << 17 | (uint32_t)(kTileRows >> 4) << 24;
}
// D (+)= A B with A in tensor memory, 16 of the summed index.  The whole warp comes
// here, so that addresses stay in uniform registers, and the lane with `lead` issues:
// with one lane on a branch of its own a product took 110 cycles to issue.
__device__ __forceinline__ void product(uint32_t d, uint32_t a, uint32_t b, uint32_t what, bool add, int lead)
{
    asm volatile("{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "setp.ne.b32 q, %6, 0;\n\t"
                 "mov.b64 b, {%2, %5};\n\t"
                 "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "r"(b), "r"(what), "r"((int)add), "r"(kOperandKind), "r"(lead)
                 : "memory");
}
// An arrival when all products issued so far are done.
__device__ __forceinline__ void products_arrive(uint32_t bar, int lead)
{
    asm volatile("{\n\t.reg .pred q;\n\t"
                 "setp.ne.b32 q, %1, 0;\n\t"
                 "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
                 "r"(lead)
                 : "memory");
}
__device__ __forceinline__ int elected()
{
    int yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes;
}

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Pairs of 32-bit numbers in one instruction.
struct Two {
    float a, b;
};
__device__ __forceinline__ Two multiply_add(uint32_t x0, uint32_t x1, float f, float d)
{
    Two y;
    asm("{\n\t.reg .b64 x, f, d;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 f, {%4, %4};\n\t"
        "mov.b64 d, {%5, %5};\n\t"
        "fma.rn.f32x2 x, x, f, d;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "=f"(y.a), "=f"(y.b) : "r"(x0), "r"(x1), "f"(f), "f"(d));
    return y;
}
__device__ __forceinline__ void add_to(Two &sum, float x0, float x1)
{
    asm("{\n\t.reg .b64 s, x;\n\t"
        "mov.b64 s, {%0, %1};\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "add.rn.f32x2 s, s, x;\n\t"
        "mov.b64 {%0, %1}, s;\n\t}"
        : "+f"(sum.a), "+f"(sum.b) : "f"(x0), "f"(x1));
}

// Largest of 32 numbers, in four chains of three-way maxima.
__device__ __forceinline__ float largest_of(const uint32_t (&x)[32])
{
    float m[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        m[c] = __uint_as_float(x[c]);
#pragma unroll
        for (int i = 4; i < 28; i += 8)
            m[c] = fmaxf(fmaxf(m[c], __uint_as_float(x[i + c])), __uint_as_float(x[i + 4 + c]));
        m[c] = fmaxf(m[c], __uint_as_float(x[28 + c]));
    }
    return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// ---- expansion ----------------------------------------------------------------------
// Pairs of 16-bit numbers, by type.
template <typename T>
struct Pair;

template <>
struct Pair<__half> {
    // u - 8 of the codes in the low four bits of each half
    static __device__ __forceinline__ uint32_t codes(uint32_t w)
    {
        uint32_t x, y;
        asm("lop3.b32 %0, %1, 0x000f000f, 0x64006400, 0xea;" : "=r"(x) : "r"(w));
        asm("add.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0xe408e408u));
        return y;
    }
    static __device__ __forceinline__ uint32_t times(uint32_t a, uint32_t b)
    {
        uint32_t y;
        asm("mul.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
        return y;
    }
    // A key's scale s = hi + lo, eight significant bits and three: times a code of up
    // to three bits both are exact, and within fp16 for s below kLarge.  An infinity's lo
    // is NaN.
    struct Key {
        uint32_t hi, lo;
    };
    static __device__ __forceinline__ Key key(uint32_t s)
    {
        Key k;
        k.hi = (s + 0x00040004u) & 0xfff8fff8u;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(k.lo) : "r"(s), "r"(k.hi));
        return k;
    }
    // both products of the codes in places c and c + 4 of a word
    static __device__ __forceinline__ void keys(uint32_t w, int c, const Key &k, uint32_t &hi, uint32_t &lo)
    {
        const uint32_t x = codes(w >> (4 * c));
        hi = times(x, k.hi);
        lo = times(x, k.lo);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t y;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
};

template <>
struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t times_add(uint32_t a, uint32_t b, uint32_t c)
    {
        uint32_t y;
        asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(a), "r"(b), "r"(c));
        return y;
    }
    static __device__ __forceinline__ uint32_t convert(uint32_t s)     // fp16 pair to bf16 pair
    {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&s));
        return pack(f.x, f.y);
    }
    // A key's scale s = hi + lo, five significant bits each (the second with a sign):
    // times a code of up to three bits both are exact, and so is either times 24.
    // (From 64544 on lo may have six, and 14 scales from 64672 on have codes whose
    // channels are rounded, by 2^-13 at most.)  NaN, of an infinity too, is in lo.
    struct Key {
        uint32_t hi, lo, hi24, lo24;        // and both times -24
    };
    static __device__ __forceinline__ Key key(uint32_t s)
    {
        Key k;
        const uint32_t h = ((__vminu2(s & 0x7fff7fffu, 0x7bdf7bdfu) + 0x00200020u) & 0xffc0ffc0u) | (s & 0x80008000u);
        uint32_t l;
        asm("sub.f16x2 %0, %1, %2;" : "=r"(l) : "r"(s), "r"(h));
        k.hi = convert(h);
        k.lo = convert(l);
        k.hi24 = times_add(k.hi, 0xc1c0c1c0u, 0x80008000u);
        k.lo24 = times_add(k.lo, 0xc1c0c1c0u, 0x80008000u);
        return k;
    }
    // Both products of the codes in places c and c + 4 of a word: a code in the upper
    // bits of the fraction of 16 makes it 16 + u, and (16 + u) s - 24 s is exact.
    static __device__ __forceinline__ void keys(uint32_t w, int c, const Key &k, uint32_t &hi, uint32_t &lo)
    {
        const uint32_t shifted = c == 0 ? w << 3 : w >> (4 * c - 3);
        uint32_t x;
        asm("lop3.b32 %0, %1, 0x00780078, 0x41804180, 0xea;" : "=r"(x) : "r"(shifted));
        hi = times_add(x, k.hi, k.hi24);
        lo = times_add(x, k.lo, k.lo24);
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        uint32_t y;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
        return y;
    }
};

// Weights 2^((s - base) c - low) of 32 scores, in fp16, and their sums.  Fine: what is left
// of each, in fp16 again.  Apart: base is not 0.
template <bool Fine, bool Apart>
__device__ __forceinline__ void weights_of(uint32_t (&w)[16], uint32_t (&rest)[Fine ? 16 : 1], const uint32_t (&s)[32],
                                           float base, float c, float low, Two (&sum)[2])
{
    sum[0] = sum[1] = Two{0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        Two y = {__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])};
        if (Apart)
            add_to(y, -base, -base);
        const Two x = multiply_add(__float_as_uint(y.a), __float_as_uint(y.b), c, -low);
        const float a = exp2_fast(x.a), b = exp2_fast(x.b);
        add_to(sum[i % 2], a, b);
        w[i] = Pair<__half>::pack(a, b);
        if (Fine) {
            float d, e;
            asm("{\n\t.reg .b16 x, y;\n\t"
                "mov.b32 {x, y}, %2;\n\t"
                "fma.rn.f32.f16 %0, x, %3, %4;\n\t"
                "fma.rn.f32.f16 %1, y, %3, %5;\n\t}"
                : "=f"(d), "=f"(e) : "r"(w[i]), "h"((unsigned short)0xbc00), "f"(a), "f"(b));
            rest[i % (Fine ? 16 : 1)] = Pair<__half>::pack(d, e);
        }
    }
}

// With fp16 queries all keys of a token that has a scale of kLarge or more (bits of an
// fp16: 4096) are taken 2^-4 times, and its scores 2^4 times: they are within fp16 then,
// and exact but for scales below 2^-10, which are rounded by 2^-21.  A key's scale is one
// of its group and place in the warp's work; lanes of a token are eight apart.  (1024
// tokens after 7168: heads of 64 301 us and 293 without, of 128 376 and 390, of 256 470
// and 460.  With a word of its own for the tokens it was 316, 392 and 469.)
constexpr unsigned kLarge = 0x6c00;
template <int Groups>
__device__ __forceinline__ unsigned lowered(const unsigned short *scales, int group, int token, unsigned long long &plain)
{
    unsigned scale = scales[group], most = scale & 0x7fffu;
    if (Groups > 4)                        // half of a token's groups are another warp's
        most = max(most, scales[group ^ 4] & 0x7fffu);
    if (__any_sync(~0u, most >= kLarge)) {
#pragma unroll
        for (int step = 8; step < 8 * Groups && step < 32; step *= 2)
            most = max(most, __shfl_xor_sync(~0u, most, step));
        if (most >= kLarge) {
            scale = __half_as_ushort(__hmul(__ushort_as_half((unsigned short)scale), __ushort_as_half(0x2c00)));
            if (group == 0)
                atomicAnd(reinterpret_cast<unsigned *>(&plain) + token / 32, ~(1u << token % 32));
        }
    }
    return scale;
}

// ---- the line of work -----------------------------------------------------------------
// One head's share of a block of rows, and the tiles [t0, t1) of tokens in it that are
// this CTA's.
struct Part {
    Block b;
    int block, head, rows, row_tiles;
    int see_lo, see_hi;        // tokens that the block's first and last row see
    int tiles, t0, t1;
    int later;                 // CTAs after this one that have tiles of it
};

// A warp's way along its CTA's places, kept in shared memory, so that what works on a
// part has the registers for itself.
struct Walk {
    Part u;
    const Block *blocks;       // all of them
    int count;
    long long x, end, per;
    int block, head;
    int more;                  // u is a part; 0: there are none left
    int pad;
};

__device__ __forceinline__ void begin(Walk &w, const Head &h, const Block *blocks, int first)
{
    w.blocks = blocks;
    w.count = h.blocks;
    w.per = h.per;
    w.x = h.per * blockIdx.x;
    w.end = w.x + h.per < h.all ? w.x + h.per : h.all;
    w.block = w.x < w.end ? first : 0;
    w.head = -1;
}

// Goes to the next part.  One thread's.
static __device__ __noinline__ void advance(const Args &p, Walk &w)
{
    const long long x = w.x, end = w.end, per = w.per;
    int block = w.block, head = w.head;
    w.more = 0;
    while (x < end && block < w.count) {
        const Block b = w.blocks[block];
        const Span s = span_of(b, p.by_group, p.group, p.rows);
        const int cost = cost_of(s);
        const long long first = b.place * p.c.kv_heads;
        if (head < 0)
            head = x > first ? (int)((x - first) / cost) : 0;
        if (head >= p.c.kv_heads) {
            ++block;
            head = 0;
            continue;
        }
        const long long at = first + (long long)head * cost;
        if (at >= end)
            break;
        auto tile_at = [&](long long place) -> int {
            const long long d = place - at - kUnitCost;
            const long long t = d <= 0 ? 0 : (d + s.weight - 1) / s.weight;
            return t < s.tiles ? (int)t : s.tiles;
        };
        Part u;
        u.b = b;
        u.block = block;
        u.head = head;
        u.rows = s.rows;
        u.row_tiles = s.row_tiles;
        u.see_lo = s.see_lo;
        u.see_hi = s.see_hi;
        u.tiles = s.tiles;
        u.t0 = p.whole ? (at >= x ? 0 : s.tiles) : tile_at(x);
        u.t1 = p.whole ? s.tiles : tile_at(end);
        u.later = 0;
        if (u.t1 > u.t0 && u.t1 < s.tiles)
            u.later = (int)((at + kUnitCost + (long long)(s.tiles - 1) * s.weight) / per) - (int)blockIdx.x;
        ++head;
        if (u.t1 > u.t0 || (s.tiles == 0 && at >= x)) {
            w.u = u;
            w.more = 1;
            break;
        }
    }
    w.block = block;
    w.head = head;
}

// What the planning launch does, by one warp for few blocks: entries a lane each,
// then blocks a lane each.
struct Few {
    Head head;
    Block blocks[kFew];
    int first;                 // block that this CTA's first place is in
};

static __device__ __noinline__ void lay_out_few(const Args &p, Few &f)
{
    const int lane = threadIdx.x & 31;
    Entry e = {};
    int start = 0, next = 0;
    if (lane < p.a.batch) {
        e = entry_of(p, lane);
        start = start_of(p, lane);
        next = start_of(p, lane + 1);
    }
    // starts as far as they rise
#pragma unroll
    for (int step = 1; step < 32; step *= 2) {
        const int y = __shfl_up_sync(~0u, start, step);
        if (lane >= step)
            start = max(start, y);
    }
    e.start = start;
    e.n = lane < p.a.batch ? max(start, next) - start : 0;
    const int count = (int)(((long long)e.n * p.group + p.rows - 1) / p.rows);
    int upto = count;
#pragma unroll
    for (int step = 1; step < 32; step *= 2) {
        const int y = __shfl_up_sync(~0u, upto, step);
        if (lane >= step)
            upto += y;
    }
    const int blocks = __shfl_sync(~0u, upto, 31);
    // block `lane`: the entry that it is of
    int owner = 0;
    for (int i = 0; i < p.a.batch; ++i)
        owner += __shfl_sync(~0u, upto, i) <= lane;
    owner = min(owner, 31);
    Block b = {};
    b.seq = __shfl_sync(~0u, e.seq, owner);
    b.start = __shfl_sync(~0u, e.start, owner);
    b.n = __shfl_sync(~0u, e.n, owner);
    b.len = __shfl_sync(~0u, e.len, owner);
    b.row0 = (lane - __shfl_sync(~0u, upto - count, owner)) * p.rows;
    const long long cost = lane < blocks ? cost_of(span_of(b, p.by_group, p.group, p.rows)) : 0;
    long long place = cost;
#pragma unroll
    for (int step = 1; step < 32; step *= 2) {
        const long long y = __shfl_up_sync(~0u, place, step);
        if (lane >= step)
            place += y;
    }
    Head h;
    h.all = __shfl_sync(~0u, place, 31) * p.c.kv_heads;
    h.per = places_of_cta(p, h.all);
    h.blocks = blocks;
    h.pad = 0;
    b.place = place - cost;
    const long long x = h.per * blockIdx.x;
    if (lane < blocks) {
        f.blocks[lane] = b;
        if (blockIdx.x == 0)
            p.blocks[lane] = b;            // for the join
        if (x >= b.place * p.c.kv_heads && x < place * p.c.kv_heads)
            f.first = lane;
    }
    if (lane == 0)
        f.head = h;
}

constexpr int kSlots = 16;     // of what is known of a tile or a unit: more than any role is ahead

struct Control {
    unsigned long long raw_full[4], raw_empty[4], key_full[4], key_empty[4], value_full[4], value_empty[4];
    unsigned long long query[2], score[2], weight[2], output[2], last;
    struct alignas(16) {
        unsigned long long there, plain;   // tokens of a tile that are there, and whose keys are as they are
    } tokens[kSlots];
    int lift[kSlots];                      // of a tile's values, a power of two
    int bad[kSlots][8];                    // of a unit: first position whose value scale is no number, a group
    uint32_t tensor;
    int lost;
    float swap[2][2][2][kTileRows];        // of a row tile's halves: maxima, sums
};

// Row r of a unit: its query's row in q and out, the query head, how many tokens it sees.
struct RowAt {
    int token, head, limit;
    __device__ __forceinline__ RowAt(const Args &p, const Part &u, int r)
    {
        const int e = u.b.row0 + (r < u.rows ? r : 0), j = p.by_group(e);
        token = u.b.start + j;
        head = u.head * p.group + (e - j * p.group);
        const int see = u.b.len - u.b.n + 1 + j;
        limit = r < u.rows && see > 0 ? see : 0;
    }
};

// First position of a part's that is there, or one beyond all.  A warp's.
static __device__ __noinline__ int first_there(const Args &p, const Part &u)
{
    const int from = u.t0 * kTokens, to = min(u.t1 * kTokens, u.see_hi), last = p.c.by_page(to - 1);
    const int32_t *row = p.c.table + u.b.seq * p.c.table_stride;
    for (int page = p.c.by_page(from); page <= last; page += 32) {
        const int mine = page + (int)(threadIdx.x & 31);
        const unsigned there = __ballot_sync(~0u, mine <= last && (unsigned)row[mine] < (unsigned)p.c.n_pages);
        if (there)
            return max(from, (page + __ffs(there) - 1) * p.c.page_size);
    }
    return 0x7fffffff;
}

// Values are multiplied by a power of two, their lift, that brings the largest scale of a
// part's first tile to [1/2, 1) (or as far as 2^15 does), and a later tile's that comes
// out at kHigh or more, so that fp16 holds what any scales make: eleven bits of those
// down to 2^-13 of the largest, and 2^-24 of that below.
constexpr unsigned kHigh = 0x6c00;          // 2^12, an fp16: times a code of 8 below 2^16
__device__ __forceinline__ int lift_of(unsigned most)
{
    const int e = 14 - (int)(most >> 10);   // most: bits of an fp16 that is finite
    return e < 15 ? e : 15;
}
__device__ __forceinline__ unsigned lift_bits(int e)      // 2^e as an fp16, e >= -16
{
    return e >= -14 ? (unsigned)(e + 15) << 10 : 0x400u >> (-14 - e);
}
// Weights are taken 2^7 times: with maxima that lag by 2^8 at most they stay within
// fp16, and 11 bits of those down to 2^-21 of the row's largest.
constexpr float kRaise = 7.f;

// Scores times c = |scale| log2 e are exponents of 2.  A row's weights are relative to a
// score, its base: to its product with c, where that is known to 2^-3, and from kFar on to
// the score itself, before the product.
constexpr float kFar = 4194304.f;
__device__ __forceinline__ float factor_of(const Args &p)
{
    // not 0, which a masked score of -inf times it would not come through, nor infinite
    return fminf(fmaxf(fabsf(p.a.scale) * kLog2e, 1.4e-45f), 3.4028234e38f);
}
// A base times c, rounded: all that is relative to it has the same rounding, which an addition
// that takes the product in would not.
__device__ __forceinline__ float scaled(float base, float c) { return __fmul_rn(base, c); }
__device__ __forceinline__ bool is_near(float m) { return fabsf(m) < kFar; }
// What a weight relative to `from` has to be taken times, for one relative to `to`.  (A
// call, as log_sum is: what is seldom run is kept out of the loops' code.)
static __device__ __noinline__ float shift_of(float from, float to, float c)
{
    const float a = scaled(from, c), b = scaled(to, c);
    const float d = is_near(a) ? (is_near(b) ? a - b : -fmaf(to, c, -a)) : (is_near(b) ? fmaf(from, c, -b) : (from - to) * c);
    return from == -INFINITY ? 0.f : exp2_fast(d);
}
// Log of a row's sum l of weights.
static __device__ __noinline__ float log_sum(const Args &p, float base, float c, float l)
{
    constexpr float kLn2 = 0.6931471805599453f;
    if (l == 0.f)
        return -INFINITY;
    const float m = scaled(base, c);
    return is_near(m) ? (m - kRaise + log2f(l)) * kLn2 : fmaf(base, fabsf(p.a.scale), (log2f(l) - kRaise) * kLn2);
}

// Small: each CTA lays few blocks out itself, where the planning launch would take as
// long as the work (one short prompt 15.2 -> 9.7 us).  A kernel of its own, since the
// code costs the loops 3 to 20 % where they run long, though it is not in them.
template <typename T, int D, bool Small>
__global__ void __launch_bounds__(Shape<D>::kThreads, 1)
chunk_kernel(const __grid_constant__ Args p)
{
    using S = Shape<D>;
    constexpr int kGroups = D / kGroup, kPer = kGroups > 4 ? 4 : kGroups;   // groups, of a stretch
    // fp16 outputs show the rounding of weights to 11 bits, so that they are two numbers
    constexpr bool kFine = std::is_same<T, __half>::value;
    extern __shared__ unsigned char smem_raw[];
    __shared__ Control ctl;
    __shared__ Walk walks[S::kThreads / 32];
    __shared__ Few few[1];
    __shared__ float bases[S::kTiles][2][kTileRows];      // each thread's own
    unsigned char *smem = smem_raw + (1024 - (shared_at(smem_raw) & 1023) & 1023);
    const int lane = threadIdx.x & 31, warp = __shfl_sync(~0u, threadIdx.x / 32, 0);

    if (threadIdx.x == 0) {
        for (int i = 0; i < 4; ++i) {
            bar_init(shared_at(&ctl.raw_full[i]), 1);
            bar_init(shared_at(&ctl.raw_empty[i]), S::kExpandWarps);
            bar_init(shared_at(&ctl.key_full[i]), S::kExpandWarps / 2);
            bar_init(shared_at(&ctl.key_empty[i]), 1);
            bar_init(shared_at(&ctl.value_full[i]), S::kExpandWarps / 2);
            bar_init(shared_at(&ctl.value_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(shared_at(&ctl.query[i]), 8);
            bar_init(shared_at(&ctl.score[i]), 1);
            bar_init(shared_at(&ctl.weight[i]), 8);
            bar_init(shared_at(&ctl.output[i]), 1);
        }
        bar_init(shared_at(&ctl.last), 1);
        ctl.lost = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x < kSlots * 8)
        ctl.bad[threadIdx.x / 8][threadIdx.x % 8] = 0x7fffffff;
    if (warp == S::kProductWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         shared_at(&ctl.tensor)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tensor = __shfl_sync(~0u, ctl.tensor, 0);
    volatile int *lost = &ctl.lost;

    dependent_grid_wait();
    allow_dependent_grid();
    if (threadIdx.x == 0 && !p.whole)
        p.splits[blockIdx.x].parts = 0;
    if (Small) {
        if (warp == 0)
            lay_out_few(p, *few);
        __syncthreads();
    }

    Walk &walk = walks[warp];
    const Part &u = walk.u;
    auto next = [&]() -> bool {        // a warp's
        __syncwarp();
        if (lane == 0)
            advance(p, walk);
        __syncwarp();
        return walk.more != 0;
    };
    if (lane == 0)
        begin(walk, Small ? few->head : *p.head, Small ? few->blocks : p.blocks,
              Small ? few->first : p.first[blockIdx.x]);

    if (warp == S::kCopyWarp) {
        // ---- records ---------------------------------------------------------------
        Turn<S::kRawStages> raw;
        int count = 0;                            // tiles so far
        const int runs = kTokens / p.run;
        while (next()) {
            const int32_t *row = p.c.table + u.b.seq * p.c.table_stride;
            const unsigned char *pool = p.c.pool + (long long)u.head * p.c.page_size * S::kRecord;
            // pages of this lane's runs (at most two) of tile t
            auto look = [&](int t, int (&page)[2]) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int pos = t * kTokens + (lane + 32 * i) * p.run;
                    page[i] = -1;
                    if (lane + 32 * i < runs && t < u.t1 && pos < u.see_hi)
                        page[i] = row[p.c.by_page(pos)];
                }
            };
            int page[2];
            look(u.t0, page);
            const int t1 = u.t1, see_hi = u.see_hi;
            for (int t = u.t0; t < t1; ++t) {
                int now[2] = {page[0], page[1]};
                look(t + 1, page);
                bar_wait(shared_at(&ctl.raw_empty[raw.stage]), raw.phase ^ 1, lost);
                const bool stop = __any_sync(~0u, *lost);
                unsigned long long there = 0;
                bool ok[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int first = (lane + 32 * i) * p.run, left = see_hi - t * kTokens - first;
                    ok[i] = (unsigned)now[i] < (unsigned)p.c.n_pages && !stop;
                    if (ok[i])
                        there |= (~0ULL >> (64 - (left < p.run ? left : p.run))) << first;
                }
                const unsigned copies = __popc(__ballot_sync(~0u, ok[0])) + __popc(__ballot_sync(~0u, ok[1]));
                const unsigned lo = __reduce_or_sync(~0u, (unsigned)there);
                const unsigned hi = __reduce_or_sync(~0u, (unsigned)(there >> 32));
                const uint32_t bar = shared_at(&ctl.raw_full[raw.stage]);
                if (lane == 0) {
                    const unsigned long long all = (unsigned long long)hi << 32 | lo;
                    ctl.tokens[count % kSlots] = {all, all};
                    if (!stop)
                        bar_expect(bar, copies * p.run * S::kRecord);
                }
                __syncwarp();
                const uint32_t to = shared_at(smem + S::kOffRaw + raw.stage * S::kRawBytes);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    if (!ok[i])
                        continue;
                    const int first = (lane + 32 * i) * p.run, pos = t * kTokens + first;
                    const int in_page = pos - p.c.by_page(pos) * p.c.page_size;
                    asm volatile(
                        "cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
                            "r"(to + first / 8 * S::kGroupBytes + first % 8 * S::kRecord),
                        "l"(pool + now[i] * p.c.page_stride + (long long)in_page * S::kRecord),
                        "r"(p.run * S::kRecord), "r"(bar)
                        : "memory");
                }
                ++count;
                raw.step();
            }
        }
        // what was started ends before the CTA does (it has, unless a wait was given up)
        if (*lost) {
            const long long from = clock_ns();
            const int n = count < S::kRawStages ? count : S::kRawStages;
            for (int i = 0; i < n; ++i) {
                const int k = count - 1 - i;
                while (!bar_done(shared_at(&ctl.raw_full[k % S::kRawStages]), k / S::kRawStages & 1) &&
                       clock_ns() - from < kPatience) {
                }
            }
        }
    } else if (warp == S::kProductWarp) {
        // ---- products ----------------------------------------------------------------------
        {
            const int lead = elected();
            Turn<S::kKeyStages> key;
            Turn<S::kValueStages> value;
            unsigned query_phase[2] = {0, 0}, weight_phase[2] = {0, 0};
            constexpr uint32_t score_kind = product_of<T>(kTokens), output_kind = product_of<__half>(D);
            const uint32_t keys = shared_at(smem + S::kOffKeys), values = shared_at(smem + S::kOffValues);
            // scores of row tile t into buffer s
            auto scores = [&](int t, int s) {
                const uint32_t d = tensor + S::kScoreColumn + s * kTokens;
                const uint32_t a = tensor + S::kQueryColumn + t * (D / 2);
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    const uint32_t b = keys + key.stage * 2 * S::kKeyBytes + part * S::kKeyBytes;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        product(d, a + k * 8, operand_at(b + k / 4 * (kTokens * 128) + k % 4 * 32), score_kind,
                                part > 0 || k > 0, lead);
                }
                products_arrive(shared_at(&ctl.score[s]), lead);
            };
            // output of row tile t, weights in buffer s
            auto outputs = [&](int t, int s, bool add) {
                const uint32_t d = tensor + S::kOutColumn + t * D, a = tensor + S::kScoreColumn + s * kTokens;
                const uint32_t b = values + value.stage * S::kValueBytes;
#pragma unroll
                for (int part = 0; part < 1 + kFine; ++part)
#pragma unroll
                    for (int k = 0; k < kTokens / 16; ++k)
                        product(d, a + part * (kTokens / 2) + k * 8, operand_at(b + k * 32), output_kind,
                                add || part > 0 || k > 0, lead);
                products_arrive(shared_at(&ctl.output[t]), lead);
            };
            auto wait_key = [&]() {
                bar_wait(shared_at(&ctl.key_full[key.stage]), key.phase, lost);
                fence_after();
                __syncwarp();
            };
            auto wait_value = [&]() {
                bar_wait(shared_at(&ctl.value_full[value.stage]), value.phase, lost);
                fence_after();
                __syncwarp();
            };
            auto wait_weight = [&](int s) {
                bar_wait(shared_at(&ctl.weight[s]), weight_phase[s], lost);
                weight_phase[s] ^= 1;
                fence_after();
                __syncwarp();
            };
            auto release_key = [&]() {
                products_arrive(shared_at(&ctl.key_empty[key.stage]), lead);
                key.step();
            };
            while (next()) {
                // the same for all lanes, which the compiler cannot know of shared memory
                const int n = __shfl_sync(~0u, u.t1 - u.t0, 0), row_tiles = __shfl_sync(~0u, u.row_tiles, 0);
                if (n == 0)
                    continue;
                for (int t = 0; t < row_tiles; ++t) {
                    bar_wait(shared_at(&ctl.query[t]), query_phase[t], lost);
                    query_phase[t] ^= 1;
                }
                if (__any_sync(~0u, *lost))
                    break;
                fence_after();
                wait_key();
                if (S::kTiles == 2 && row_tiles == 2) {
                    scores(0, 0);
                    scores(1, 1);
                    release_key();
                    for (int j = 0; j < n; ++j) {
                        wait_value();
                        wait_weight(0);
                        outputs(0, 0, j > 0);
                        if (j + 1 < n) {
                            wait_key();
                            scores(0, 0);
                        }
                        wait_weight(1);
                        outputs(1, 1, j > 0);
                        if (j + 1 < n)
                            scores(1, 1);
                        products_arrive(shared_at(&ctl.value_empty[value.stage]), lead);
                        value.step();
                        if (j + 1 < n)
                            release_key();
                    }
                } else {
                    // one row tile: the buffers take turns, scores a product ahead
                    scores(0, 0);
                    release_key();
                    for (int j = 0; j < n; ++j) {
                        if (j + 1 < n) {
                            wait_key();
                            scores(0, (j + 1) % 2);
                            release_key();
                        }
                        wait_value();
                        wait_weight(j % 2);
                        outputs(0, j % 2, j > 0);
                        products_arrive(shared_at(&ctl.value_empty[value.stage]), lead);
                        value.step();
                    }
                }
            }
            // nothing is under way when tensor memory is given back
            products_arrive(shared_at(&ctl.last), lead);
            const long long from = clock_ns();
            while (!bar_done(shared_at(&ctl.last), 0) && clock_ns() - from < kPatience) {
            }
        }
        __syncwarp();
    } else if (warp >= S::kExpandWarp && warp % 4 >= 2) {
        // ---- values: V^T, a row for each channel -----------------------------------------
        Turn<S::kRawStages> raw;
        Turn<S::kValueStages> value;
        int count = 0, unit = 0;
        const int turn = ((warp - S::kExpandWarp) / 4 * 2 + warp % 4 - 2) * 32 + lane;
        while (next()) {
            if (u.t1 == u.t0)
                continue;
            // the slot of a unit to come, which no one looks at any more: expansion
            // is at most kValueStages units ahead, row tiles one apart
            if (turn < 8)
                ctl.bad[(unit + kSlots / 2) % kSlots][turn] = 0x7fffffff;
            int *bad = ctl.bad[unit++ % kSlots];
            int lift = 0;
            bool fresh = true;
            const int t1 = u.t1, see_lo = u.see_lo;
            for (int t = u.t0; t < t1; ++t) {
                bar_wait(shared_at(&ctl.raw_full[raw.stage]), raw.phase, lost);
                bar_wait(shared_at(&ctl.value_empty[value.stage]), value.phase ^ 1, lost);
                const unsigned char *src = smem + S::kOffRaw + raw.stage * S::kRawBytes;
                unsigned char *dst = smem + S::kOffValues + value.stage * S::kValueBytes;
                const unsigned long long there = ctl.tokens[count % kSlots].there;
                const bool masked = there != ~0ULL || (t + 1) * kTokens > see_lo;
                // a lane's work: eight tokens of one word, which is four channels of two
                // neighbouring groups
                constexpr int kWords = D / 8;
                static_assert(kWords * 8 <= S::kExpandThreads, "a word a lane");
                const int eight = turn % 8, word = turn / 8, place = word % (4 * kPer) * 2;
                const int g = place / kPer, group = word / (4 * kPer) * kPer + place % kPer;
                const unsigned char *rec = src + eight * S::kGroupBytes;
                if (masked && word < kWords) {
                    // Tokens that are not there, or that not every row sees, may hold
                    // anything: their weights are 0, which 0 * NaN is not.  Their scales
                    // are put right in place; other lanes may do the same.
                    const unsigned here = (unsigned)(there >> (8 * eight)) & 255;
#pragma unroll 1
                    for (int k = 0; k < 8; ++k) {
                        uint32_t *scales = reinterpret_cast<uint32_t *>(const_cast<unsigned char *>(rec) + k * S::kRecord + D + D / 16 + group * 2);
                        const uint32_t given = here >> k & 1 ? *scales : 0u;
                        uint32_t fine = given;
                        const int pos = t * kTokens + 8 * eight + k;
                        if ((given & 0x7c00u) == 0x7c00u) {
                            atomicMin(&bad[group], pos);
                            fine &= 0xffff0000u;
                        }
                        if ((given & 0x7c000000u) == 0x7c000000u) {
                            atomicMin(&bad[group + 1], pos);
                            fine &= 0xffffu;
                        }
                        *scales = fine;
                    }
                }
                __syncwarp();
                uint32_t s[8];
                unsigned high = 0;
                if (word < kWords) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const unsigned char *scales = rec + k * S::kRecord + D + D / 16;
                        s[k] = *reinterpret_cast<const uint32_t *>(scales + group * 2);
                        high = __vmaxu2(high, s[k]);
                        if (kGroups > kPer)        // the other stretch's, which is other warps' work
                            high = __vmaxu2(high, *reinterpret_cast<const uint32_t *>(scales + (group ^ kPer) * 2));
                    }
                }
                // Every warp that has work meets all scales in some lane, so that all of
                // these come to the same lift.  Against kHigh exponents are compared, of
                // what may not be there, or no number, too: then it is looked at again.
                if (__any_sync(~0u, fresh || (int)(max(high & 0xffffu, high >> 16) >> 10) + lift >= (int)(kHigh >> 10))) {
                    unsigned most = 0;
#pragma unroll 1
                    for (int k = 0; k < 2; ++k) {
                        const int token = lane + 32 * k;
                        const unsigned short *scales = reinterpret_cast<const unsigned short *>(
                            src + token / 8 * S::kGroupBytes + token % 8 * S::kRecord + D + D / 16);
#pragma unroll 1
                        for (int g = 0; g < kGroups; ++g) {
                            const unsigned x = scales[g] & 0x7fffu;
                            if ((there >> token & 1) && x < 0x7c00u)
                                most = max(most, x);
                        }
                    }
                    most = __reduce_max_sync(~0u, most);
                    if (fresh || (int)(most >> 10) + lift >= (int)(kHigh >> 10))
                        lift = lift_of(most);
                    fresh = false;
                }
                const unsigned lift2 = lift_bits(lift) * 0x10001u;
                if (turn == 0)
                    ctl.lift[count % kSlots] = lift;
                if (word < kWords) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        w[k] = *reinterpret_cast<const uint32_t *>(rec + k * S::kRecord + D / 2 + word * 4);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const unsigned pick = half ? 0x7632 : 0x5410;
                        uint32_t x[4], f[4];
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                            x[m] = __byte_perm(w[2 * m], w[2 * m + 1], pick);
                            f[m] = Pair<__half>::times(__byte_perm(s[2 * m], s[2 * m + 1], pick), lift2);
                        }
                        const int channel = (group + half) * kGroup + 4 * g;
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int d = channel + c;
                            uint4 v;
                            v.x = Pair<__half>::times(Pair<__half>::codes(x[0] >> (4 * c)), f[0]);
                            v.y = Pair<__half>::times(Pair<__half>::codes(x[1] >> (4 * c)), f[1]);
                            v.z = Pair<__half>::times(Pair<__half>::codes(x[2] >> (4 * c)), f[2]);
                            v.w = Pair<__half>::times(Pair<__half>::codes(x[3] >> (4 * c)), f[3]);
                            *reinterpret_cast<uint4 *>(dst + d * 128 + ((eight ^ (d & 7)) * 16)) = v;
                        }
                    }
                }
                fence_proxy();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(shared_at(&ctl.raw_empty[raw.stage]));
                    bar_arrive(shared_at(&ctl.value_full[value.stage]));
                }
                ++count;
                raw.step();
                value.step();
            }
        }
    } else if (warp >= S::kExpandWarp) {
        // ---- keys: a row for each token ----------------------------------------------------
        Turn<S::kRawStages> raw;
        Turn<S::kKeyStages> key;
        int count = 0;
        const int turn = ((warp - S::kExpandWarp) / 4 * 2 + warp % 4) * 32 + lane;
        while (next()) {
            const int t1 = u.t1;
            for (int t = u.t0; t < t1; ++t) {
                bar_wait(shared_at(&ctl.raw_full[raw.stage]), raw.phase, lost);
                bar_wait(shared_at(&ctl.key_empty[key.stage]), key.phase ^ 1, lost);
                const unsigned char *src = smem + S::kOffRaw + raw.stage * S::kRawBytes;
                unsigned char *dst = smem + S::kOffKeys + key.stage * 2 * S::kKeyBytes;
#pragma unroll 1
                for (int i = turn; i < kTokens * kGroups; i += S::kExpandThreads) {
                    // a group of one token: four words
                    const int token = i / (8 * kGroups) * 8 + i % 8, group = i / 8 % kGroups;
                    const int stretch = group / kPer, g = group % kPer;
                    const unsigned char *rec = src + token / 8 * S::kGroupBytes + token % 8 * S::kRecord;
                    const uint32_t *words = reinterpret_cast<const uint32_t *>(rec + stretch * 64) + g;
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        w[k] = words[k * kPer];
                    const unsigned short *scales = reinterpret_cast<const unsigned short *>(rec + D);
                    const unsigned scale =
                        kFine ? lowered<kGroups>(scales, group, token, ctl.tokens[count % kSlots].plain) : scales[group];
                    const typename Pair<T>::Key key_scale = Pair<T>::key(scale * 0x10001u);
                    const int piece = stretch * 16 + 4 * g;               // of eight channels, the first
                    unsigned char *row = dst + piece / 8 * (kTokens * 128) + token * 128;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        unsigned char *at = row + (((piece + k) & 7) ^ (token & 7)) * 16;
                        uint4 x, y;
                        Pair<T>::keys(w[k], 0, key_scale, x.x, y.x);
                        Pair<T>::keys(w[k], 1, key_scale, x.y, y.y);
                        Pair<T>::keys(w[k], 2, key_scale, x.z, y.z);
                        Pair<T>::keys(w[k], 3, key_scale, x.w, y.w);
                        *reinterpret_cast<uint4 *>(at) = x;
                        *reinterpret_cast<uint4 *>(at + S::kKeyBytes) = y;
                    }
                }
                fence_proxy();
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(shared_at(&ctl.raw_empty[raw.stage]));
                    bar_arrive(shared_at(&ctl.key_full[key.stage]));
                }
                ++count;
                raw.step();
                key.step();
            }
        }
    } else {
        // ---- softmax: half a row a thread ------------------------------------------------------
        const int tile = warp / 8, half = warp / 4 % 2, local = warp % 4 * 32 + lane;
        const uint32_t rows_at = tensor + ((uint32_t)(warp % 4 * 32) << 16);
        const int r = tile * kTileRows + local;
        const uint32_t out_at = rows_at + S::kOutColumn + tile * D + half * (D / 2);
        unsigned score_phase[2] = {0, 0}, output_phase = 0, side = 0;
        // The other half's value for this row, where both warps of the rows meet.
        // Past it both have their scores, whose columns either's weights go to.
        auto meet = [&]() -> float {
            fence_before();
            asm volatile("bar.sync %0, 64;" ::"r"(1 + tile * 4 + warp % 4) : "memory");
            fence_after();
            const float y = ctl.swap[side][tile][half ^ 1][local];
            side ^= 1;
            return y;
        };
        Turn<S::kValueStages> value;
        int count = 0, unit = 0;
        const float c = factor_of(p);
        const uint32_t flip = p.a.scale < 0.f ? 0x80008000u : 0u;
        while (next()) {
            const int n = u.t1 - u.t0, slot = unit % kSlots;
            unit += n > 0;
            if (S::kTiles == 2)       // one tile's warps are at most a unit ahead of the other's
                asm volatile("bar.sync 9, 512;" ::: "memory");
            const bool ahead = u.row_tiles == 1;      // the buffers take turns
            if (tile >= u.row_tiles) {
                // what happened without these warps
                count += n;
                for (int t = 0; t < n; ++t)
                    value.step();
                score_phase[0] ^= (n + 1) / 2 & 1;
                score_phase[1] ^= n / 2 & 1;
                continue;
            }
            if (!ahead)
                score_phase[tile ^ 1] ^= n & 1;
            int spin = tile;                          // the buffer of the next scores
            const bool in = r < u.rows;
            const int limit = RowAt(p, u, r).limit;
            // What the row's weights are relative to is seldom looked at, and kept in shared
            // memory; m is its product with c where that is near, else -inf.
            bases[tile][half][local] = -INFINITY;
            float m = -INFINITY, l = 0.f;
            int lift = 0;              // that the output has
            if (n > 0) {
                // the row's query, channels (j, j + 4) of each eight in pairs
                const RowAt row(p, u, r);
                const T *q = (const T *)p.a.q + row.token * p.a.q_query + row.head * p.a.q_head;
#pragma unroll 1
                for (int part = 0; part < D / 64; ++part) {
                    const int first = half * (D / 2) + part * 32;
                    uint4 v[4] = {};
                    if (in && p.q_vector) {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = *reinterpret_cast<const uint4 *>(q + first + e * 8);
                    } else if (in) {
                        const unsigned short *y = reinterpret_cast<const unsigned short *>(q + first);
#pragma unroll
                        for (int e = 0; e < 4; ++e, y += 8)
                            v[e] = make_uint4(y[0] | (unsigned)y[1] << 16, y[2] | (unsigned)y[3] << 16,
                                              y[4] | (unsigned)y[5] << 16, y[6] | (unsigned)y[7] << 16);
                    }
                    uint32_t x[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        x[4 * e] = __byte_perm(v[e].x, v[e].z, 0x5410) ^ flip;
                        x[4 * e + 1] = __byte_perm(v[e].x, v[e].z, 0x7632) ^ flip;
                        x[4 * e + 2] = __byte_perm(v[e].y, v[e].w, 0x5410) ^ flip;
                        x[4 * e + 3] = __byte_perm(v[e].y, v[e].w, 0x7632) ^ flip;
                    }
                    __syncwarp();
                    store_columns(rows_at + S::kQueryColumn + tile * (D / 2) + first / 2, x);
                }
                wait_stores();
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(shared_at(&ctl.query[tile]));
            }
            const int t0 = u.t0, t1 = u.t1, see_lo = u.see_lo;
            for (int t = t0; t < t1; ++t) {
                const uint32_t at = rows_at + S::kScoreColumn + spin * kTokens;
                // The lift is known when the values are expanded, which is mostly before the
                // scores are there.  With one stage of values it is not, and is waited for when
                // the weights are worked out (D = 256 410 us for 437; the others 6 to 10 % slower).
                constexpr bool kLate = S::kValueStages == 1;
                int lift_now = 0;
                if (!kLate) {
                    bar_wait(shared_at(&ctl.value_full[value.stage]), value.phase, lost);
                    value.step();
                    lift_now = ctl.lift[count % kSlots];
                }
                // With fp16 queries keys are looked at, too, which are expanded when the scores
                // are there.
                constexpr bool kEarly = !kLate && !kFine;
                const unsigned *known = reinterpret_cast<const unsigned *>(&ctl.tokens[count % kSlots]) + half;
                unsigned there = 0;
                if (kEarly)
                    there = *known;
                ++count;
                bar_wait(shared_at(&ctl.score[spin]), score_phase[spin], lost);
                score_phase[spin] ^= 1;
                fence_after();
                __syncwarp();
                if (!kEarly)
                    there = known[kFine ? 2 : 0];
                uint32_t s[32];
                load_columns(s, at + half * 32);
                wait_loads();
                if (there != ~0u || (t + 1) * kTokens > see_lo) {
                    if constexpr (kFine) {
                        const unsigned plain = there;
                        there = *known;
                        if (there != plain) {
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                s[i] = (there & ~plain) >> i & 1 ? __float_as_uint(__uint_as_float(s[i]) * 16.f) : s[i];
                        }
                    }
                    const int left = limit - t * kTokens - half * 32;
                    const unsigned see = there & (left >= 32 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - left));
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        s[i] = see >> i & 1 ? s[i] : 0xff800000u;
                }
                // Weights are relative to a maximum that follows the true one only where
                // that is 8 above it, which is seldom: they are worked out before the other
                // half's maximum is known, and again where it turns out that it grows, or
                // that the row is far from 0.
                float most = largest_of(s);
                ctl.swap[side][tile][half][local] = most;
                Two sum[2];
                uint32_t w[16], rest[kFine ? 16 : 1];
                weights_of<kFine, false>(w, rest, s, 0.f, c, (m == -INFINITY ? 0.f : m) - kRaise, sum);
                if (kLate) {
                    bar_wait(shared_at(&ctl.value_full[value.stage]), value.phase, lost);
                    value.step();
                    lift_now = ctl.lift[(count - 1) % kSlots];
                }
                most = fmaxf(most, meet());
                const bool grows = most * c > m + 8.f || (m == -INFINITY && most > -INFINITY);
                if (__any_sync(~0u, grows || lift_now != lift)) {
                    const float from = bases[tile][half][local], base = (most - from) * c > 8.f ? most : from;
                    float f = shift_of(from, base, c);
                    l *= f;
                    bases[tile][half][local] = base;
                    m = scaled(base, c);
                    const bool near = is_near(m) || base == -INFINITY;
                    m = near ? m : -INFINITY;
                    f *= __uint_as_float((unsigned)(lift_now - lift + 127) << 23);
                    lift = lift_now;
                    if (t > t0) {
                        bar_wait(shared_at(&ctl.output[tile]), output_phase ^ 1, lost);
                        fence_after();
                        __syncwarp();
#pragma unroll 1
                        for (int part = 0; part < D / 2; part += 16) {
                            uint32_t x[16];
                            load_columns(x, out_at + part);
                            wait_loads();
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            store_columns(out_at + part, x);
                        }
                    }
                    weights_of<kFine, true>(w, rest, s, near ? 0.f : base, c, (m == -INFINITY ? 0.f : m) - kRaise,
                                            sum);
                }
                store_columns(at + half * 16, w);
                if constexpr (kFine)
                    store_columns(at + kTokens / 2 + half * 16, rest);
                l += (sum[0].a + sum[1].a) + (sum[0].b + sum[1].b);
                wait_stores();
                // With one row tile scores are a product ahead of outputs.  The output
                // before this one ends before these weights are given away, so that never
                // two phases of its barrier are to come, which a parity could not tell.
                if (ahead && t > t0)
                    bar_wait(shared_at(&ctl.output[tile]), output_phase ^ 1, lost);
                fence_before();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(shared_at(&ctl.weight[spin]));
                output_phase ^= 1;
                if (ahead)
                    spin ^= 1;
            }
            // ---- the unit's end
            const bool whole = n == u.tiles;
            float *partial = nullptr;
            if (!whole) {
                partial = p.partial + (2LL * blockIdx.x + (u.t0 == 0)) * S::kPartial;
                if (u.t0 == 0 && r == 0 && half == 0) {
                    p.splits[blockIdx.x].block = u.block;
                    p.splits[blockIdx.x].head = u.head;
                    p.splits[blockIdx.x].parts = 1 + u.later;
                }
            }
            if (n > 0) {
                ctl.swap[side][tile][half][local] = l;
                l += meet();
                bar_wait(shared_at(&ctl.output[tile]), output_phase ^ 1, lost);
                fence_after();
                __syncwarp();
            }
            // No weight at all: nothing was seen, or all scores were -inf, as an infinite
            // query's may be, which gives NaN.  For the join that is a sum of -0.
            const bool none = l == 0.f && limit > u.t0 * kTokens;
            if (__any_sync(~0u, none)) {
                const int first = first_there(p, u);
                if (none && limit > first)
                    l = whole ? __uint_as_float(0x7fffffffu) : -0.f;
            }
            float base = bases[tile][half][local];
            const float down = __uint_as_float((unsigned)(127 - lift) << 23);
            float inv = l == 0.f ? 0.f : down / l;
            if (*lost)
                inv = l = base = __uint_as_float(0x7fffffffu);
            const RowAt row(p, u, r);
            const long long to = (long long)row.token * p.a.heads + row.head;
#pragma unroll 1
            for (int part = half * (D / 2); part < (half + 1) * (D / 2); part += 32) {
                uint32_t x[32];
                __syncwarp();
                if (n > 0) {
                    load_columns(x, rows_at + S::kOutColumn + tile * D + part);
                    wait_loads();
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = 0;
                }
                const bool nan = n > 0 && limit > ctl.bad[slot][part / 32];
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        partial[(part + i) * S::kRows + r] = nan ? __uint_as_float(0x7fffffffu) : __uint_as_float(x[i]) * down;
                } else if (in) {
                    const float f = nan ? __uint_as_float(0x7fffffffu) : inv;
                    // rows that see nothing are 0, whatever the tile before left there
                    uint32_t y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        y[i] = f == 0.f ? 0u : Pair<T>::pack(__uint_as_float(x[2 * i]) * f, __uint_as_float(x[2 * i + 1]) * f);
                    uint4 *dst = reinterpret_cast<uint4 *>((T *)p.a.out + to * D + part);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        dst[i] = make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                }
            }
            if (half != 0) {
                // the other half's
            } else if (!whole) {
                partial[D * S::kRows + r] = base;
                partial[(D + 1) * S::kRows + r] = l;
            } else if (in && p.a.lse) {
                p.a.lse[to] = log_sum(p, base, c, l);
            }
            fence_before();
        }
    }

    __syncthreads();
    if (warp == S::kProductWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tensor));
}

// Joins the parts of the unit that begins in a CTA and goes on in others: 32 of its
// rows, a row a lane, the channels shared out between the warps.
constexpr int kJoinThreads = 256;

template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads)
join_chunk_kernel(const __grid_constant__ Args p)
{
    using S = Shape<D>;
    constexpr int kMine = D / (kJoinThreads / 32), kSlices = S::kRows / 32;
    dependent_grid_wait();
    allow_dependent_grid();
    const int cta = blockIdx.x / kSlices, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const Split s = p.splits[cta];
    if (s.parts == 0)
        return;
    const Block b = p.blocks[s.block];
    const Span span = span_of(b, p.by_group, p.group, p.rows);
    const int r = (blockIdx.x - cta * kSlices) * 32 + lane;
    if (r - lane >= span.rows)
        return;
    auto part_at = [&](int i) { return p.partial + (2LL * (cta + i) + (i == 0)) * S::kPartial; };
    const float c = factor_of(p);
    float base = -INFINITY;
    for (int i = 0; i < s.parts; ++i)
        base = fmaxf(base, part_at(i)[D * S::kRows + r]);
    float l = 0.f, x[kMine];
    bool seen = false;             // something that had no weight
#pragma unroll
    for (int k = 0; k < kMine; ++k)
        x[k] = 0.f;
    for (int i = 0; i < s.parts; ++i) {
        const float *q = part_at(i);
        const float from = q[D * S::kRows + r], pl = q[(D + 1) * S::kRows + r];
        float v[kMine];
#pragma unroll
        for (int k = 0; k < kMine; ++k)
            v[k] = q[(warp * kMine + k) * S::kRows + r];
        const float w = shift_of(from, base, c);
        l += pl * w;
        seen = seen || __float_as_uint(pl) == 0x80000000u;
#pragma unroll
        for (int k = 0; k < kMine; ++k)
            x[k] = fmaf(v[k], w, x[k]);
    }
    if (r >= span.rows)
        return;
    Part u;
    u.b = b;
    u.head = s.head;
    u.rows = span.rows;
    const RowAt row(p, u, r);
    const long long to = (long long)row.token * p.a.heads + row.head;
    if (l == 0.f && seen)
        l = __uint_as_float(0x7fffffffu);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t y[kMine / 2];
#pragma unroll
    for (int k = 0; k < kMine / 2; ++k)
        y[k] = Pair<T>::pack(x[2 * k] * inv, x[2 * k + 1] * inv);
    uint4 *dst = reinterpret_cast<uint4 *>((T *)p.a.out + to * D + warp * kMine);
#pragma unroll
    for (int k = 0; k < kMine / 8; ++k)
        dst[k] = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
    if (warp == 0 && p.a.lse)
        p.a.lse[to] = log_sum(p, base, c, l);
}

template <int D>
cudaError_t launch_chunk_dim(const Args &p, int dev, int ctas, cudaStream_t stream)
{
    using S = Shape<D>;
    auto fn = p.a.bf16 ? (p.few ? chunk_kernel<__nv_bfloat16, D, true> : chunk_kernel<__nv_bfloat16, D, false>)
                       : (p.few ? chunk_kernel<__half, D, true> : chunk_kernel<__half, D, false>);
    auto join = p.a.bf16 ? join_chunk_kernel<__nv_bfloat16, D> : join_chunk_kernel<__half, D>;
    static std::atomic<unsigned long long> raised[4];       // the kernels' shared memory, once a device
    const int which = 2 * p.few + p.a.bf16;
    cudaError_t e = cudaSuccess;
    if (!(raised[which].load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
        if (e != cudaSuccess)
            return e;
        raised[which].fetch_or(1ULL << dev, std::memory_order_relaxed);
    }
    e = launch_overlapped(fn, ctas, S::kThreads, S::kSmem, stream, p);
    if (e != cudaSuccess || p.whole)
        return e;
    return launch_overlapped(join, ctas * (S::kRows / 32), kJoinThreads, 0, stream, p);
}

}  // namespace chunk
}  // namespace kv4
}  // namespace ds
