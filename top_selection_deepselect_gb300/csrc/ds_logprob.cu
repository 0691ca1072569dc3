// ds_logprob.cu -- log probabilities of given tokens with entropy and the
// likeliest alternatives, and their gradient (include/ds_logprob.h).
//
// Forward, one pass over a row: with a running maximum m of the logits,
//   S = sum 2^d,  T = sum 2^d d,  d = x c - m c,  c = scale log2 e
// give lse = scale m + ln S and entropy = ln 2 (log2 S - T / S), whose two terms
// are both >= 0, so that nothing cancels.  m c is rounded once, which shifts all d
// alike: that drops out of the entropy and is taken back in lse, as long as m c is below
// 2^22 and 2^d near 1 for the maximum itself.  Logits of -inf are
// lifted to a lowest finite one, whose 2^d is 0, so that 2^d d is 0 and not NaN.  For
// that no maximum is taken from logits as low as that, masks of the type's lowest value
// for one: until another comes sums are relative to 0, which such logits add nothing to.
// Where the maximum is too near to the lowest, or too large, the row is summed again
// with the difference taken first.
//
// The alternatives come out of the same pass: the first vectors of a CTA's slice
// give a value that at least k of its logits reach; where a later vector's largest
// is above it, the vector's number goes to a list.  At the end the logits of the
// listed vectors that reach the value are taken out again, and the k first of these
// by (value, index) are found by warps that sort and merge lists of 32.
//
// The bound is HBM; what has to be kept off is instructions and waits.  A lane
// copies its vectors of 16 bytes to shared memory asynchronously, kDepth ahead, and
// reads only its own, so that no barrier is needed; a vector is tested as a whole, by
// packed maxima, against the value that candidates have to be above (which is at or
// below the running maximum), so that maxima and candidates cost next to nothing;
// products and sums are pairs in one instruction.
//
// A row is a CTA's, or a cluster's where rows are few: each CTA takes a slice, and
// the first joins the sums and the sorted lists out of distributed shared memory.
#include "ds_logprob.h"

#include <cooperative_groups.h>
#include <type_traits>

#include "ds_device.cuh"
#include "ds_host.h"
#include "ds_kv4.cuh"

namespace ds {
namespace logprob {
namespace {

using kv4::from_float;
using kv4::to_float;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
// Vectors of a thread under way; as many give the first bound.  2048 x 128000 112 us, with
// four 119; 512 x 128000 fp32 with 20 alternatives 75, with four 184 (twice the candidates).
constexpr int kDepth = 8;
constexpr int kTop = DS_LOGPROB_MAX_K;
constexpr int kEach = kTop / kWarps;   // of a warp's threads that the first bound is taken from
constexpr int kCapacity = 1024;    // listed vectors of a slice, and candidates among their logits
constexpr float kLow = -200.f;     // 2^d is 0 in 32 bits below -150
constexpr float kLog2e = 1.4426950408889634f;
constexpr double kLn2 = 0.6931471805599453;

// Key of the value, then 2^31 - 1 - index: larger comes first.  None is ~0, and 0 is none.
typedef unsigned long long Entry;

template <typename T>
struct alignas(16) Vec {
    static constexpr int kCount = 16 / sizeof(T);
    T x[kCount];
};

__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Maxima that keep a NaN.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ __half2 max_nan(__half2 a, __half2 b) { return __hmax2_nan(a, b); }
__device__ __forceinline__ __nv_bfloat162 max_nan(__nv_bfloat162 a, __nv_bfloat162 b)
{
    return __hmax2_nan(a, b);
}

// Largest element of a vector, NaN if there is one.
__device__ __forceinline__ float largest(const Vec<float> &v)
{
    return max_nan(max_nan(v.x[0], v.x[1]), max_nan(v.x[2], v.x[3]));
}
template <typename T, typename T2>
__device__ __forceinline__ float largest16(const Vec<T> &v)
{
    const T2 *w = reinterpret_cast<const T2 *>(v.x);
    const T2 m = max_nan(max_nan(w[0], w[1]), max_nan(w[2], w[3]));
    return max_nan(to_float(m.x), to_float(m.y));
}
__device__ __forceinline__ float largest(const Vec<__half> &v) { return largest16<__half, __half2>(v); }
__device__ __forceinline__ float largest(const Vec<__nv_bfloat16> &v)
{
    return largest16<__nv_bfloat16, __nv_bfloat162>(v);
}

// Unsigned key in the order of values: NaN above +inf, -0 equal to +0.
__device__ __forceinline__ unsigned key_of(float x)
{
    if (x != x)
        return ~0u;
    const unsigned b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(unsigned key)
{
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);   // the NaN's key gives a NaN
}

// A row as vectors of 16 aligned bytes: element i is element i + skip of them.
template <typename T>
struct Row {
    const T *at;                  // aligned address at or below the row's start
    unsigned skip, past;          // the row is elements [skip, past) from there
    unsigned vectors;
    __device__ __forceinline__ Row(const T *row, int vocab)
    {
        const uintptr_t a = (uintptr_t)row;
        skip = (unsigned)(a % 16 / sizeof(T));
        at = reinterpret_cast<const T *>(a & ~(uintptr_t)15);
        past = skip + (unsigned)vocab;
        vectors = (past + Vec<T>::kCount - 1) / Vec<T>::kCount;
    }
    __device__ __forceinline__ bool whole(unsigned j) const
    {
        return j * Vec<T>::kCount >= skip && (j + 1) * Vec<T>::kCount <= past;
    }
    // Element e of vector j, -inf in the places that are not the row's.
    __device__ __forceinline__ T element(unsigned j, int e) const
    {
        const unsigned i = j * Vec<T>::kCount + e;
        T x;
        from_float(x, -INFINITY);
        return i >= skip && i < past ? at[i] : x;
    }
    __device__ __forceinline__ Vec<T> load(unsigned j, unsigned end) const
    {
        Vec<T> v;
        if (j < end && whole(j)) {
            v = *reinterpret_cast<const Vec<T> *>(at + (size_t)j * Vec<T>::kCount);
        } else {
#pragma unroll
            for (int e = 0; e < Vec<T>::kCount; ++e)
                v.x[e] = element(j < end ? j : 0xfffffff0u / Vec<T>::kCount, e);
        }
        return v;
    }
};

// Sums of a thread, a CTA or a row: pairs of partial sums, by parity of the place.
struct Sums {
    float most;                   // maximum so far (not a NaN); -inf: nothing but -inf so far
    float s0, s1, t0, t1;
};

// A difference of logits in powers of 2.  scale log2 e may be beyond 32 bits where
// this is not.
__device__ __forceinline__ float exponent(float d, float scale) { return max_nan(d * scale * kLog2e, kLow); }

// Brings sums to another maximum at or above theirs.
__device__ __forceinline__ void rescale(Sums &a, float most, float scale)
{
    if (a.most == -INFINITY) {    // then the sums are 0, or a NaN's
        a.most = most;
        return;
    }
    const float d = exponent(a.most - most, scale), f = exp2_fast(d);
    a.t0 = f * fmaf(d, a.s0, a.t0), a.t1 = f * fmaf(d, a.s1, a.t1);
    a.s0 *= f, a.s1 *= f;
    a.most = most;
}

__device__ __forceinline__ void add_sums(Sums &a, Sums b, float scale)
{
    const float most = fmaxf(a.most, b.most);
    rescale(a, most, scale);
    rescale(b, most, scale);
    a.s0 += b.s0, a.s1 += b.s1, a.t0 += b.t0, a.t1 += b.t1;
}

// Adds two elements, relative to base (a.most, or 0 while that is -inf).
__device__ __forceinline__ void add_pair(Sums &a, float x0, float x1, float base, float scale)
{
    const float d0 = exponent(x0 - base, scale), d1 = exponent(x1 - base, scale);
    const float e0 = exp2_fast(d0), e1 = exp2_fast(d1);
    asm("{\n\t.reg .b64 s, t, e, d;\n\t"
        "mov.b64 s, {%0, %1};\n\t"
        "mov.b64 t, {%2, %3};\n\t"
        "mov.b64 e, {%4, %5};\n\t"
        "mov.b64 d, {%6, %7};\n\t"
        "add.rn.f32x2 s, s, e;\n\t"
        "fma.rn.f32x2 t, e, d, t;\n\t"
        "mov.b64 {%0, %1}, s;\n\t"
        "mov.b64 {%2, %3}, t;\n\t}"
        : "+f"(a.s0), "+f"(a.s1), "+f"(a.t0), "+f"(a.t1) : "f"(e0), "f"(e1), "f"(d0), "f"(d1));
}

template <typename T>
__device__ __forceinline__ void add_vector(Sums &a, const Vec<T> &v, float scale)
{
    const float base = a.most == -INFINITY ? 0.f : a.most;
#pragma unroll
    for (int e = 0; e < Vec<T>::kCount; e += 2)
        add_pair(a, to_float(v.x[e]), to_float(v.x[e + 1]), base, scale);
}

// ---- lists of 32 entries, one a lane, largest first ----------------------------
template <typename K>
__device__ __forceinline__ K exchange(K x, int step, bool larger)
{
    const K y = __shfl_xor_sync(~0u, x, step);
    return larger == (x > y) ? x : y;
}

// The larger half of a bitonic sequence's sort, largest first.
template <typename K>
__device__ __forceinline__ K order_bitonic(K x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int step = 16; step; step /= 2)
        x = exchange(x, step, (lane & step) == 0);
    return x;
}

template <typename K>
__device__ __forceinline__ K order_lanes(K x)
{
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size < 32; size *= 2)
#pragma unroll
        for (int step = size / 2; step; step /= 2)
            x = exchange(x, step, ((lane & step) == 0) == ((lane & size) == 0));
    return order_bitonic(x);
}

// The 32 largest of two lists.
__device__ __forceinline__ Entry merge_lists(Entry a, Entry b)
{
    const Entry r = __shfl_sync(~0u, b, 31 - (threadIdx.x & 31));
    return order_bitonic(a > r ? a : r);
}

// The 32 largest of n entries, in warp 0 (in all warps of the first call's
// threads, something).  `lists`: kWarps * 32 entries of shared memory.
__device__ Entry select_entries(const Entry *entries, int n, Entry *lists)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    Entry mine = 0;
    for (int i = warp * 32; i < n; i += kThreads)
        mine = merge_lists(mine, order_lanes(i + lane < n ? entries[i + lane] : 0));
#pragma unroll
    for (int half = kWarps / 2; half; half /= 2) {
        if (warp >= half && warp < 2 * half)
            lists[warp * 32 + lane] = mine;
        __syncthreads();
        if (warp < half)
            mine = merge_lists(mine, lists[(warp + half) * 32 + lane]);
    }
    return mine;
}

struct Shared {
    Entry entries[kCapacity];
    unsigned vectors[kCapacity];
    Entry lists[kWarps * 32];
    Sums sums[kWarps];
    unsigned keys[kWarps * kEach];
    float most[kWarps];
    int listed, count;
    // what the cluster's first CTA reads
    Entry top[kTop];
    Sums all;
};

template <typename T>
__device__ __forceinline__ Entry entry_of(const Row<T> &row, T x, unsigned j, int e)
{
    return (Entry)key_of(to_float(x)) << 32 | (0x7fffffffu - (j * Vec<T>::kCount + e - row.skip));
}

__device__ __forceinline__ void keep(Shared &sh, Entry x)
{
    const int at = atomicAdd(&sh.count, 1);
    if (at < kCapacity)
        sh.entries[at] = x;
}

// The 32 largest entries of the slice where candidates did not fit: the k-th
// largest of the threads' largest is a bound that k entries reach, and mostly few
// more do; where those do not fit either, entry after entry is found by a
// sweep.  In warp 0.
template <typename T>
__device__ __noinline__ Entry select_slowly(const Row<T> &row, unsigned lo, unsigned hi, int k, Shared &sh)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    // the thread's largest entry below `under`
    auto largest_below = [&](Entry under) {
        Entry most = 0;
        for (unsigned j = lo + threadIdx.x; j < hi; j += kThreads) {
            const Vec<T> v = row.load(j, hi);
#pragma unroll
            for (int e = 0; e < Vec<T>::kCount; ++e) {
                const unsigned i = j * Vec<T>::kCount + e;
                const Entry x = entry_of(row, v.x[e], j, e);
                if (i >= row.skip && i < row.past && x < under && x > most)
                    most = x;
            }
        }
        return most;
    };
    __syncthreads();
    static_assert(kThreads <= kCapacity, "an entry of each thread");
    sh.entries[threadIdx.x] = largest_below(~0ULL);
    __syncthreads();
    Entry mine = select_entries(sh.entries, kThreads, sh.lists);
    __syncthreads();
    if (warp == 0) {
        const Entry bound = __shfl_sync(~0u, mine, k - 1);
        if (lane == 0) {
            sh.top[0] = bound;
            sh.count = 0;
        }
    }
    __syncthreads();
    const Entry bound = sh.top[0];
    for (unsigned j = lo + threadIdx.x; j < hi; j += kThreads) {
        const Vec<T> v = row.load(j, hi);
#pragma unroll
        for (int e = 0; e < Vec<T>::kCount; ++e) {
            const unsigned i = j * Vec<T>::kCount + e;
            const Entry x = entry_of(row, v.x[e], j, e);
            if (i >= row.skip && i < row.past && x >= bound)
                keep(sh, x);
        }
    }
    __syncthreads();
    if (sh.count <= kCapacity)
        return select_entries(sh.entries, sh.count, sh.lists);
    Entry found = ~0ULL;
    mine = 0;
    for (int n = 0; n < k; ++n) {
        Entry most = largest_below(found);
#pragma unroll
        for (int step = 16; step; step /= 2) {
            const Entry y = __shfl_xor_sync(~0u, most, step);
            most = y > most ? y : most;
        }
        __syncthreads();
        if (lane == 0)
            sh.lists[warp] = most;
        __syncthreads();
        found = sh.lists[0];
        for (int w = 1; w < kWarps; ++w)
            found = sh.lists[w] > found ? sh.lists[w] : found;
        if (lane == n)
            mine = found;
    }
    return mine;
}

struct Args {
    const void *logits;
    long long stride;
    const int32_t *tokens;
    float *logprob, *entropy, *lse, *top;
    int32_t *idx;
    int vocab, k, cluster;
    float scale;
};

// Waits until all but the newest n groups of this thread's copies have ended.
template <int n>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

// Products of a maximum and c that are rounded by 2^-3 at most.
constexpr float kFar = 4194304.f;

// What the fast sums take a maximum from is above this: above what logits of -inf, and
// lower ones, are lifted to (-65504 with fp16 and -1e30 otherwise), and not so far below 0
// that the rounding of m c would show in 2^d.
template <typename T>
__device__ __forceinline__ float floor_of(float c)
{
    return fmaxf(std::is_same<T, __half>::value ? -65504.f : -1e29f, -kFar / c);
}

// Pairs of floats, in 64-bit registers so that what does not change is paired once.
typedef unsigned long long Two;
__device__ __forceinline__ Two pair(float a, float b)
{
    Two y;
    asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(a), "f"(b));
    return y;
}
__device__ __forceinline__ void apart(Two x, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ Two times_add(Two x, Two y, Two z)
{
    Two r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ Two sum(Two x, Two y)
{
    Two r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}

// Adds a vector to sums s and t of terms relative to -mc2 = m c.
__device__ __forceinline__ void add_two(Two &s, Two &t, float x0, float x1, Two mc2, Two c2)
{
    const Two d = times_add(pair(x0, x1), c2, mc2);
    float d0, d1;
    apart(d, d0, d1);
    const Two e = pair(exp2_fast(d0), exp2_fast(d1));
    s = sum(s, e);
    t = times_add(e, d, t);
}
__device__ __forceinline__ void add_fast(Two &s, Two &t, const Vec<float> &v, Two mc2, Two c2)
{
    constexpr float low = -1e30f;
    add_two(s, t, max_nan(v.x[0], low), max_nan(v.x[1], low), mc2, c2);
    add_two(s, t, max_nan(v.x[2], low), max_nan(v.x[3], low), mc2, c2);
}
__device__ __forceinline__ void add_fast(Two &s, Two &t, const Vec<__half> &v, Two mc2, Two c2)
{
    const __half2 low2 = __half2half2(__ushort_as_half(0xfbff));     // -65504
    const __half2 *w = reinterpret_cast<const __half2 *>(v.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(max_nan(w[i], low2));
        add_two(s, t, x.x, x.y, mc2, c2);
    }
}
__device__ __forceinline__ void add_fast(Two &s, Two &t, const Vec<__nv_bfloat16> &v, Two mc2, Two c2)
{
    const unsigned *w = reinterpret_cast<const unsigned *>(v.x);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        unsigned x;                                                  // lifted to -1e30
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(x) : "r"(w[i]), "r"(0xf14af14au));
        add_two(s, t, __uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u), mc2, c2);
    }
}

// Of a maximum: m c, and 0 for one that there is not yet.
__device__ __forceinline__ float scaled(float most, float c) { return most == -INFINITY ? 0.f : most * c; }

// Brings fast sums to another maximum at or above theirs.
__device__ __forceinline__ void lift_fast(Sums &a, float most, float c)
{
    const float d = scaled(a.most, c) - scaled(most, c);
    if (a.most != -INFINITY) {               // else the sums are 0, or a NaN's
        const float f = exp2_fast(fmaxf(d, -1000.f));
        a.t0 = f * fmaf(d, a.s0, a.t0), a.t1 = f * fmaf(d, a.s1, a.t1);
        a.s0 *= f, a.s1 *= f;
    }
    a.most = most;
}
__device__ __forceinline__ void join_fast(Sums &a, Sums b, float c)
{
    const float most = fmaxf(a.most, b.most);
    lift_fast(a, most, c);
    lift_fast(b, most, c);
    a.s0 += b.s0, a.s1 += b.s1, a.t0 += b.t0, a.t1 += b.t1;
}

__device__ __forceinline__ Sums shuffled(const Sums &a, int step)
{
    Sums b;
    b.most = __shfl_xor_sync(~0u, a.most, step);
    b.s0 = __shfl_xor_sync(~0u, a.s0, step), b.s1 = __shfl_xor_sync(~0u, a.s1, step);
    b.t0 = __shfl_xor_sync(~0u, a.t0, step), b.t1 = __shfl_xor_sync(~0u, a.t1, step);
    return b;
}

// Sums of vectors [lo, hi) by the CTA, differences taken first, in every thread.
template <typename T>
__device__ __noinline__ Sums sum_carefully(const Row<T> &row, unsigned lo, unsigned hi, float scale, Sums *sums)
{
    Sums a = {-INFINITY, 0.f, 0.f, 0.f, 0.f};
    for (unsigned j = lo + threadIdx.x; j < hi; j += kThreads) {
        const Vec<T> v = row.load(j, hi);
        float most = a.most;
#pragma unroll
        for (int e = 0; e < Vec<T>::kCount; ++e)
            most = fmaxf(most, to_float(v.x[e]));
        if (most > a.most)
            rescale(a, most, scale);
        add_vector(a, v, scale);
    }
#pragma unroll
    for (int step = 16; step; step /= 2)
        add_sums(a, shuffled(a, step), scale);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        sums[threadIdx.x / 32] = a;
    __syncthreads();
    a = sums[0];
    for (int w = 1; w < kWarps; ++w)
        add_sums(a, sums[w], scale);
    return a;
}

// 2048 x 128000 bf16: 112 us alone, 97 in turn (5.4 TB/s, 81 % of the measured copy rate),
// issue slots 73 % busy: some 63 instructions for eight logits, 26 of them for the sums
// themselves.  256 x 128000 with 20 alternatives 25 us in turn.  Loads to registers, four
// ahead, took 304 and 69: the lanes' waits, not HBM.  Two or four vectors a step 116 and
// 114 where one took 115; five CTAs an SM the same.
template <typename T>
__global__ void __launch_bounds__(kThreads, 4)
logprob_kernel(const __grid_constant__ Args p)
{
    __shared__ Shared sh;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    Vec<T> *ring = reinterpret_cast<Vec<T> *>(ring_bytes) + threadIdx.x;     // slot i at i * kThreads
    dependent_grid_wait();
    allow_dependent_grid();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const unsigned r = blockIdx.x / p.cluster, rank = blockIdx.x - r * p.cluster;
    const T *logits = (const T *)p.logits + (long long)r * p.stride;
    const Row<T> row(logits, p.vocab);
    const unsigned lo = (unsigned)((unsigned long long)row.vectors * rank / p.cluster);
    const unsigned hi = (unsigned)((unsigned long long)row.vectors * (rank + 1) / p.cluster);
    const float c = p.scale * kLog2e;

    // The slice's whole vectors [from, to), a thread's kThreads apart, in rounds of kDepth.
    // Past them a slot holds -inf, which adds nothing.
    const unsigned from = max(lo, row.skip ? 1u : 0u), to = max(from, min(hi, row.past / Vec<T>::kCount));
    unsigned j = from + threadIdx.x;
    const T *source = row.at + (size_t)j * Vec<T>::kCount;
    Vec<T> none;
#pragma unroll
    for (int e = 0; e < Vec<T>::kCount; ++e)
        from_float(none.x[e], -INFINITY);
    const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
    auto fetch = [&](int i, int turn) {        // the vector `turn` ahead to slot i
        if (j + turn * kThreads < to)
            cp_async16(ring_at + i * kThreads * 16, source + turn * kThreads * Vec<T>::kCount);
        else
            ring[i * kThreads] = none;
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        fetch(i, i);
    if (threadIdx.x == 0)
        sh.listed = sh.count = 0;
    // The row's first and last vector, where they are not whole, are two threads' besides.
    unsigned ragged = ~0u;
    if (threadIdx.x == 0 && lo < from && lo < hi)
        ragged = lo;
    if (threadIdx.x == 1 && hi > to && hi - 1 >= from)
        ragged = hi - 1;
    const Vec<T> edge = row.load(ragged, hi);

    // The first vectors: their maximum, which all sums start from, and a value that k
    // of their logits reach.
    cp_async_wait<0>();
    float mine = -INFINITY;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
        const float m = largest(ring[i * kThreads]);
        nan = nan || m != m;
        mine = fmaxf(mine, m);
    }
    const unsigned mine_key = nan ? ~0u : key_of(mine);
#pragma unroll
    for (int e = 0; e < Vec<T>::kCount; ++e)
        mine = fmaxf(mine, to_float(edge.x[e]));
    const unsigned top_key = __reduce_max_sync(~0u, key_of(mine));
    if (lane == 0)
        sh.most[warp] = value_of(top_key);
    if (p.k > 0) {
        // four largest of each warp's threads, and the k-th of these; a thread
        // of places outside the row has -inf, which is at or below all logits
        const unsigned sorted = order_lanes(mine_key);
        if (lane < kEach)
            sh.keys[warp * kEach + lane] = sorted;
    }
    __syncthreads();
    mine = sh.most[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
        mine = fmaxf(mine, sh.most[w]);
    // A listed vector's largest has to be above `bound`; among the first ones at it, too:
    // above the value before it.  (An equal one further on comes later in the order.)  The
    // vectors at the row's ends are listed anyhow.
    float bound = mine, reach = mine;
    if (p.k > 0) {
        const unsigned key = __shfl_sync(~0u, order_lanes(sh.keys[lane]), p.k - 1);
        reach = value_of(key);
        bound = value_of(key == 0x80000000u ? key - 2 : key - 1);     // 0 has no other sign below it
    }

    const float floor = floor_of<T>(c);
    Sums a = {mine > floor ? mine : -INFINITY, 0.f, 0.f, 0.f, 0.f};
    Two sums = 0, weighted = 0;
    Two mc2 = pair(-scaled(a.most, c), -scaled(a.most, c));
    const Two c2 = pair(c, c);
    auto list = [&](unsigned at) {
        const int n = atomicAdd(&sh.listed, 1);
        if (n < kCapacity)
            sh.vectors[n] = at;
    };
    const unsigned rounds = (to - from + kDepth * kThreads - 1) / (kDepth * kThreads);
#pragma unroll 1
    for (unsigned round = 0; round < rounds; ++round) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            cp_async_wait<kDepth - 1>();
            const Vec<T> v = ring[i * kThreads];
            const float m = largest(v);
            if (!(m <= bound)) {
                if (p.k > 0 && j + i * kThreads < to)
                    list(j + i * kThreads);
                float most = fmaxf(a.most, m);
                if (m != m) {
#pragma unroll 1
                    for (int e = 0; e < Vec<T>::kCount; ++e)
                        most = fmaxf(most, to_float(ring[i * kThreads].x[e]));
                }
                if (most > a.most && most > floor) {
                    apart(sums, a.s0, a.s1);
                    apart(weighted, a.t0, a.t1);
                    lift_fast(a, most, c);
                    sums = pair(a.s0, a.s1);
                    weighted = pair(a.t0, a.t1);
                    mc2 = pair(-scaled(most, c), -scaled(most, c));
                }
            }
            add_fast(sums, weighted, v, mc2, c2);
            fetch(i, kDepth + i);
        }
        j += kDepth * kThreads;
        source += kDepth * kThreads * Vec<T>::kCount;
        bound = reach;
    }
    if (ragged != ~0u) {
        add_fast(sums, weighted, edge, mc2, c2);
        if (p.k > 0)
            list(ragged);
    }
    cp_async_wait<0>();
    apart(sums, a.s0, a.s1);
    apart(weighted, a.t0, a.t1);

    // the CTA's sums, in a fixed order
#pragma unroll
    for (int step = 16; step; step /= 2)
        join_fast(a, shuffled(a, step), c);
    if (lane == 0)
        sh.sums[warp] = a;
    __syncthreads();
    a = sh.sums[0];
    for (int w = 1; w < kWarps; ++w)
        join_fast(a, sh.sums[w], c);
    // Sums of what the fast form cannot tell from a logit of -inf, or overflows on, are
    // made again; and all sums are relative to the maximum itself from here on.
    const bool fine = (a.most - floor) * c >= 150.f && a.most * c < kFar && a.most < 1e29f && c <= 1e8f;
    if (fine) {
        const float mc = scaled(a.most, c), off = fmaf(a.most, c, -mc), f = exp2f(-off);
        a.t0 = f * fmaf(-off, a.s0, a.t0), a.t1 = f * fmaf(-off, a.s1, a.t1);
        a.s0 *= f, a.s1 *= f;
    } else {
        a = sum_carefully(row, lo, hi, p.scale, sh.sums);
    }
    Entry best = 0;
    if (p.k > 0) {
        // the logits of the listed vectors that reach the value
        const int listed = sh.listed;
        for (int i = threadIdx.x; i < listed && listed <= kCapacity; i += kThreads) {
            const unsigned at = sh.vectors[i];
            const Vec<T> v = row.load(at, hi);
#pragma unroll
            for (int e = 0; e < Vec<T>::kCount; ++e) {
                const unsigned place = at * Vec<T>::kCount + e;
                if (!(to_float(v.x[e]) < reach) && place >= row.skip && place < row.past)
                    keep(sh, entry_of(row, v.x[e], at, e));
            }
        }
        __syncthreads();
        best = listed <= kCapacity && sh.count <= kCapacity ? select_entries(sh.entries, sh.count, sh.lists)
                                                            : select_slowly(row, lo, hi, p.k, sh);
    }
    if (p.cluster > 1 && warp == 0) {
        sh.top[lane] = best;
        if (lane == 0)
            sh.all = a;
    }
    if (p.cluster > 1) {
        namespace cg = cooperative_groups;
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        if (rank == 0 && warp == 0)
            for (int other = 1; other < p.cluster; ++other) {
                const Shared *far = cluster.map_shared_rank(&sh, other);
                add_sums(a, far->all, p.scale);
                if (p.k > 0)
                    best = merge_lists(best, far->top[lane]);
            }
        cluster.sync();           // the others' shared memory lives until it was read
    }
    if (rank != 0 || warp != 0)
        return;
    const float s = a.s0 + a.s1, t = a.t0 + a.t1;
    const float bits = log2f(s);                     // of the sum
    const bool empty = s == 0.f;                     // nothing but -inf
    auto log_prob = [&](float x) {       // of a logit
        return empty ? -INFINITY : (float)(((double)x - a.most) * p.scale - kLn2 * bits);
    };
    if (lane == 0) {
        p.lse[r] = empty ? -INFINITY : (float)((double)p.scale * a.most + kLn2 * bits);
        p.entropy[r] = empty ? 0.f : (float)(kLn2 * (double)(bits - t / s));
        const int token = p.tokens[r];
        p.logprob[r] = (unsigned)token < (unsigned)p.vocab ? log_prob(to_float(logits[token])) : 0.f;
    }
    if (lane < p.k) {
        const long long at = (long long)r * p.k + lane;
        p.idx[at] = (int)(0x7fffffffu - (unsigned)best);
        p.top[at] = log_prob(value_of((unsigned)(best >> 32)));
    }
}

// ---- gradient --------------------------------------------------------------------
// dz_i = p_i (g_lse - g_logprob - sum g_top - g_entropy (log p_i + entropy)), plus
// the token's and the alternatives' own gradients in their places, which are
// written again by one thread each after the CTA's pass.  One read and one write
// of the row, a CTA for each piece of it: 1024 x 128000 bf16 102 us (5.1 TB/s, 77 % of
// the measured copy rate), waiting for loads.  Two vectors ahead of the work 140 us,
// four 220, because of the registers; loads past L1 105.
struct GradArgs {
    const void *logits;
    void *grad;
    long long stride, grad_stride;
    const int32_t *tokens, *idx;
    const float *lse, *entropy, *g_logprob, *g_entropy, *g_lse, *g_top;
    int vocab, k, pieces;
    unsigned each;                // vectors of a piece
    float scale;
};

template <typename T>
__device__ __forceinline__ float exponential(float x)
{
    // 16-bit results: the fast exponential's 2^-22 is far below their rounding
    return sizeof(T) == 4 ? expf(x) : exp2_fast(x * kLog2e);
}

// log p = (x - base) scale - lse: base is 0, or the row's maximum where lse is so
// large that its rounding would show in p.
struct Factors {
    float scale, base, lse, common, g_entropy, entropy;
    bool empty;
};

template <typename T>
__device__ __forceinline__ float slope(const Factors &f, float x)
{
    const float logp = fmaf(x - f.base, f.scale, -f.lse);
    const float prob = exponential<T>(logp);
    const float g = prob * (f.common - f.g_entropy * (logp + f.entropy));
    return prob == 0.f || f.empty ? 0.f : g;
}

// lse is summed again from here on.  p is off by its half unit in the last place,
// relative: with 32-bit results up to 2^-19 below 64, little more than what log p is
// rounded by; results of 16 bits show nothing below 1024, where it is 2^-15.  The sum
// reads the row once more for each of its pieces: 8 x 128000 fp32 83 us where 9 without,
// 1024 x 50257 122 where 79 (so that 32, 2^-20, is not worth it).
template <typename T>
__device__ __forceinline__ float large()
{
    return sizeof(T) == 4 ? 64.f : 1024.f;
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads)
gradient_kernel(const __grid_constant__ GradArgs p)
{
    __shared__ int place[kTop + 1];
    __shared__ float share[kTop + 1];
    __shared__ Sums sums[kWarps];
    dependent_grid_wait();
    allow_dependent_grid();
    const int lane = threadIdx.x & 31;
    const unsigned r = blockIdx.x / p.pieces, piece = blockIdx.x - r * p.pieces;
    const T *logits = (const T *)p.logits + (long long)r * p.stride;
    T *grad = (T *)p.grad + (long long)r * p.grad_stride;
    const Row<T> row(logits, p.vocab);
    const unsigned lo = piece * p.each, hi = lo + p.each < row.vectors ? lo + p.each : row.vectors;

    const int token = p.tokens[r];
    const bool given = (unsigned)token < (unsigned)p.vocab;
    const float g_logprob = p.g_logprob && given ? p.g_logprob[r] : 0.f;
    float g_top = 0.f;
    int top_at = -1;
    if (lane < p.k) {
        top_at = p.idx[(long long)r * p.k + lane];
        if ((unsigned)top_at < (unsigned)p.vocab)
            g_top = p.g_top[(long long)r * p.k + lane];
        else
            top_at = -1;
    }
    float sum = g_top;
#pragma unroll
    for (int step = 16; step; step /= 2)
        sum += __shfl_xor_sync(~0u, sum, step);
    Factors f;
    f.scale = p.scale;
    f.lse = p.lse[r];
    f.base = 0.f;
    f.empty = false;
    f.entropy = p.entropy[r];
    f.g_entropy = p.g_entropy ? p.g_entropy[r] : 0.f;
    f.common = (p.g_lse ? p.g_lse[r] : 0.f) - g_logprob - sum;

    // the token and the alternatives: their logits are read before anything of
    // the row is written, which may be in their place
    float own = 0.f;
    int at = -1;
    if (threadIdx.x <= (unsigned)p.k) {
        at = threadIdx.x < (unsigned)p.k ? top_at : given ? token : -1;
        place[threadIdx.x] = at;
        share[threadIdx.x] = threadIdx.x < (unsigned)p.k ? g_top : g_logprob;
        if (at >= 0)
            own = to_float(logits[at]);
    }
    if (fabsf(f.lse) >= large<T>()) {
        const Sums a = sum_carefully(row, 0, row.vectors, f.scale, sums);
        f.empty = a.s0 + a.s1 == 0.f;
        f.base = f.empty ? 0.f : a.most;
        f.lse = (float)(kLn2 * (double)log2f(a.s0 + a.s1));
    }
    __syncthreads();

    for (unsigned j = lo + threadIdx.x; j < hi; j += kThreads) {
        const Vec<T> v = row.load(j, hi);
        Vec<T> out;
#pragma unroll
        for (int e = 0; e < Vec<T>::kCount; ++e)
            from_float(out.x[e], slope<T>(f, to_float(v.x[e])) * f.scale);
        const long long first = (long long)j * Vec<T>::kCount - row.skip;
        if (kVec && row.whole(j)) {
            *reinterpret_cast<Vec<T> *>(grad + first) = out;
        } else {
#pragma unroll
            for (int e = 0; e < Vec<T>::kCount; ++e)
                if (first + e >= 0 && first + e < p.vocab)
                    grad[first + e] = out.x[e];
        }
    }
    __syncthreads();
    if (at >= 0) {
        const unsigned j = (at + row.skip) / Vec<T>::kCount;
        bool mine = j >= lo && j < hi;
        for (int i = 0; i < (int)threadIdx.x; ++i)
            mine = mine && place[i] != at;             // the first of equal ones
        if (mine) {
            float g = slope<T>(f, own);
            for (int i = threadIdx.x; i <= p.k; ++i)
                if (place[i] == at)
                    g += share[i];
            if (f.empty)
                g = 0.f;
            from_float(grad[at], g * f.scale);
        }
    }
}

// CTAs of a row: one where rows alone fill the GPU twice, else as many as give slices of
// at least kSlice vectors a thread.  8 x 128000 17.5 us in clusters of eight, 25.8 in one
// CTA a row; 256 rows 32 in clusters of two, 32 in one, 40 in clusters of four.
constexpr int kSlice = 8;

template <typename T>
cudaError_t launch_forward(Args &p, long long rows, int sms, cudaStream_t stream)
{
    p.cluster = 1;
    const long long vectors = (p.vocab + Vec<T>::kCount - 1) / Vec<T>::kCount;
    while (p.cluster < 8 && rows * p.cluster < 2LL * sms &&
           vectors >= 2LL * p.cluster * kSlice * kThreads)
        p.cluster *= 2;
    return launch_clusters(logprob_kernel<T>, p.cluster, (unsigned)(rows * p.cluster), kThreads,
                           kDepth * kThreads * 16, stream, p);
}

template <typename T>
cudaError_t launch_gradient(GradArgs &p, long long rows, int sms, cudaStream_t stream)
{
    const long long vectors = (p.vocab + 2LL * Vec<T>::kCount - 2) / Vec<T>::kCount;   // at most
    // Four CTAs an SM: with 16, pieces of 257 x 50257 are three vectors a thread, and take
    // 34 us instead of 30; with two, 36.  In its own place a row is one CTA's, which may
    // have to read it twice.
    long long pieces = 1;
    while (p.grad != p.logits && rows * pieces < 4LL * sms && vectors > pieces * kThreads * 2)
        pieces *= 2;
    p.each = (unsigned)((vectors + pieces - 1) / pieces);
    p.pieces = (int)pieces;
    const size_t size = sizeof(T);
    // rows of the gradient start where those of the logits do within 16 bytes
    const bool vec = (uintptr_t)p.grad % 16 == (uintptr_t)p.logits % 16 &&
                     (rows < 2 || p.grad_stride * size % 16 == p.stride * size % 16);
    auto fn = vec ? gradient_kernel<T, true> : gradient_kernel<T, false>;
    return launch_overlapped(fn, (unsigned)(rows * pieces), kThreads, 0, stream, p);
}

int check(const void *logits, int dtype, int64_t rows, int64_t vocab, int64_t stride, const int32_t *tokens,
          int k, float scale)
{
    if (dtype != DS_FP32 && dtype != DS_BF16 && dtype != DS_FP16)
        return fail(DS_EUNSUPPORTED, "dtype %d is not DS_FP32 (0), DS_BF16 (1) or DS_FP16 (2)", dtype);
    if (rows < 0 || vocab < 1)
        return fail(DS_EINVAL, "rows = %lld must be >= 0 and vocab = %lld >= 1", (long long)rows,
                    (long long)vocab);
    if (vocab >= DS_LOGPROB_MAX_VOCAB || rows >= 1LL << 27)
        return fail(DS_EUNSUPPORTED, "rows = %lld and vocab = %lld must be below 2^27 and 2^31 - 64",
                    (long long)rows, (long long)vocab);
    if (rows > 1 && stride < vocab)
        return fail(DS_EINVAL, "row_stride = %lld is below vocab = %lld", (long long)stride, (long long)vocab);
    if (k < 0 || k > vocab)
        return fail(DS_EINVAL, "k = %d must be >= 0 and at most vocab = %lld", k, (long long)vocab);
    if (k > DS_LOGPROB_MAX_K)
        return fail(DS_EUNSUPPORTED, "k = %d is above %d", k, DS_LOGPROB_MAX_K);
    if (!(scale > 0.f) || !(scale < INFINITY))
        return fail(DS_EINVAL, "scale = %g must be finite and above 0", scale);
    if (rows == 0)
        return DS_OK;
    if (!logits || !tokens)
        return fail(DS_EINVAL, "logits and tokens must be non-NULL when rows > 0");
    if ((uintptr_t)logits % (dtype == DS_FP32 ? 4 : 2) != 0)
        return fail(DS_EINVAL, "logits must be aligned to its elements");
    return DS_OK;
}

}  // namespace
}  // namespace logprob
}  // namespace ds

extern "C" {

int ds_token_logprobs(const void *logits, int dtype, int64_t rows, int64_t vocab,
                      int64_t row_stride, const int32_t *tokens, int k, float scale,
                      float *logprob, float *entropy, float *lse, int32_t *idx, float *top,
                      void *stream)
{
    using namespace ds::logprob;
    ds::g_detail[0] = '\0';
    int dev = 0, sms = 0, rc = check(logits, dtype, rows, vocab, row_stride, tokens, k, scale);
    if (rc != DS_OK || rows == 0)
        return rc;
    if (!logprob || !entropy || !lse || (k > 0 && (!idx || !top)))
        return ds::fail(DS_EINVAL, "logprob, entropy and lse, and with k > 0 idx and top, must be non-NULL");
    if ((rc = ds::current_device(&dev, &sms)) != DS_OK)
        return rc;
    Args p = {logits, row_stride, tokens, logprob, entropy, lse, top, idx, (int)vocab, k, 1, scale};
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == DS_FP32   ? launch_forward<float>(p, rows, sms, s)
                          : dtype == DS_BF16 ? launch_forward<__nv_bfloat16>(p, rows, sms, s)
                                             : launch_forward<__half>(p, rows, sms, s);
    return e == cudaSuccess ? DS_OK : ds::fail_cuda(e, "ds_token_logprobs");
}

int ds_token_logprobs_backward(const void *logits, int dtype, int64_t rows, int64_t vocab,
                               int64_t row_stride, const int32_t *tokens, int k,
                               const int32_t *idx, float scale, const float *lse,
                               const float *entropy, const float *grad_logprob,
                               const float *grad_entropy, const float *grad_lse,
                               const float *grad_top, void *grad, int64_t grad_stride,
                               void *stream)
{
    using namespace ds::logprob;
    ds::g_detail[0] = '\0';
    int dev = 0, sms = 0, rc = check(logits, dtype, rows, vocab, row_stride, tokens, k, scale);
    if (rc != DS_OK)
        return rc;
    if (rows > 1 && grad_stride < vocab)
        return ds::fail(DS_EINVAL, "grad_stride = %lld is below vocab = %lld", (long long)grad_stride,
                        (long long)vocab);
    if (rows == 0)
        return DS_OK;
    if (!lse || !entropy || !grad || (grad_top && k > 0 && !idx))
        return ds::fail(DS_EINVAL, "lse, entropy and grad, and with grad_top idx, must be non-NULL");
    if ((uintptr_t)grad % (dtype == DS_FP32 ? 4 : 2) != 0)
        return ds::fail(DS_EINVAL, "grad must be aligned to its elements");
    if ((rc = ds::current_device(&dev, &sms)) != DS_OK)
        return rc;
    GradArgs p = {logits, grad, row_stride, grad_stride, tokens, idx, lse, entropy, grad_logprob,
                  grad_entropy, grad_lse, grad_top, (int)vocab, grad_top ? k : 0, 1, 0, scale};
    const cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = dtype == DS_FP32   ? launch_gradient<float>(p, rows, sms, s)
                          : dtype == DS_BF16 ? launch_gradient<__nv_bfloat16>(p, rows, sms, s)
                                             : launch_gradient<__half>(p, rows, sms, s);
    return e == cudaSuccess ? DS_OK : ds::fail_cuda(e, "ds_token_logprobs_backward");
}

}  // extern "C"
