// ds_kv4_store.cu -- append to and read from the 4-bit cache.
//
// One lane holds eight channels of one token's key or value (16 bytes of a
// 16-bit type), so a vector of D channels takes D/8 neighbouring lanes and a
// group of 32 channels four of them: the group's largest magnitude is two
// shuffles away, and the reordering inside the record is a shuffle too, so that
// codes leave and arrive as whole words.  Both kernels move each byte once and
// are bound by the bytes only while a lane's eight channels cost few
// instructions, so that magnitudes are compared as bits, quotients and integers
// come from multiply-adds, and nothing is divided per lane but by constants.
#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct alignas(sizeof(T) * 8 < 16 ? sizeof(T) * 8 : 16) Eight {
    T x[8];
};

// What a lane works on: rows of D/8 lanes are (token, head, key or value), the
// last fastest.
template <int D>
struct Place {
    int token, head, which, w, slot;
    bool in;
    __device__ __forceinline__ Place(const Cache &c, const Divider &by_heads,
                                     const int32_t *__restrict__ seq, const int32_t *__restrict__ pos,
                                     int tokens)
    {
        w = threadIdx.x % (D / 8);
        // rows / 2 is below 2^31: the callers refuse more
        const long long row = (long long)blockIdx.x * (kThreads / (D / 8)) + threadIdx.x / (D / 8);
        which = (int)(row & 1);
        const int r = (int)(row >> 1);
        token = by_heads(r);
        head = r - token * c.kv_heads;
        in = token < tokens;
        slot = in ? token_slot(c, __ldg(seq + token), __ldg(pos + token)) : -1;
    }
};

// Lane (of the D/8 lanes of a vector) whose word holds what stored word p of
// a key starts with, and its inverse: words of a stretch are stored with word
// 4 i + t at place n t + i.
template <int D>
__device__ __forceinline__ int key_source(int p)
{
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    return (p & ~(4 * n - 1)) | 4 * (p % n) | (p / n % 4);
}
template <int D>
__device__ __forceinline__ int key_place(int w)
{
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    return (w & ~(4 * n - 1)) | n * (w % 4) | (w / 4 % n);
}

// x / step rounded to the nearest float, step normal or subnormal fp16 and inv
// the nearest float to 1 / step: the quotient's first value is within one unit
// in the last place, and one correction by the exact remainder makes it the
// nearest (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Dev. 34, 1990).  A rounded quotient is
// what the format asks for: ties of x / scale go to even.
__device__ __forceinline__ float quotient(float x, float step, float inv)
{
    const float q = x * inv;
    return fmaf(fmaf(-q, step, x), inv, q);
}

template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(kThreads)
append_kernel(Cache c, Divider by_heads, const int32_t *__restrict__ seq,
              const int32_t *__restrict__ pos, int tokens, const T *__restrict__ k, long long k_token,
              long long k_head, const T *__restrict__ v, long long v_token, long long v_head)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);
    const Place<D> at(c, by_heads, seq, pos, tokens);
    float x[8];
    if (at.slot >= 0) {
        const T *src = at.which ? v + at.token * v_token + at.head * v_head
                                : k + at.token * k_token + at.head * k_head;
        if (kVec) {
            const Eight<T> e = *reinterpret_cast<const Eight<T> *>(src + at.w * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = to_float(e.x[j]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = to_float(src[at.w * 8 + j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = 0.f;
    }

    // largest magnitude of the group: bits of magnitudes are in their order,
    // those that are not finite above all others
    unsigned most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        most = max(most, __float_as_uint(x[j]) & 0x7fffffffu);
    most = max(most, __shfl_xor_sync(~0u, most, 1));
    most = max(most, __shfl_xor_sync(~0u, most, 2));
    const bool bad = most >= 0x7f800000u;      // a NaN or an infinity poisons the group
    __half scale = __float2half_rn(__uint_as_float(most) / 7.f);
    if (__hisinf(scale))
        scale = __ushort_as_half(0x7bff);
    const float step = __half2float(scale);
    // zero, subnormal and largest scales: codes may be anything or beyond 7
    const bool edge = step < 6.103515625e-05f || step == 65504.f;
    const float inv = step > 0.f ? 1.f / step : 0.f;
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        q[j] = quotient(x[j], step, inv);
    if (edge) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            q[j] = fminf(fmaxf(q[j], -7.f), 7.f);
    }
    // the float q + 12582920 (1.5 2^23 + 8) holds rint(q) + 8 in its low
    // bits, above a constant that the sum takes away once for all eight
    unsigned word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        word += __float_as_uint(q[j] + 12582920.f) << (4 * j);
    word -= 0x3f400000u;
    word = bad || step == 0.f ? 0x88888888u : word;
    const unsigned bits = bad ? 0x7fffu : __half_as_ushort(scale);

    // stored order
    const unsigned kw = __shfl_sync(~0u, word, first + key_source<D>(at.w));
    // value: word p holds pieces (g, i) and (g, i + 1), n g + i = 2 p within
    // the stretch; piece (g, i) is half g & 1 of word 4 i + g / 2
    const int local = at.w & (4 * n - 1), g = 2 * local / n, i = 2 * local % n;
    const int from = first + (at.w & ~(4 * n - 1)) + g / 2 + 4 * i;
    const unsigned lo = __shfl_sync(~0u, word, from), hi = __shfl_sync(~0u, word, from + 4);
    const unsigned vw = __byte_perm(lo, hi, g & 1 ? 0x7632 : 0x5410);
    // scales: four lanes of a group hold it; neighbours (4 i, 4 i + 4) pair up
    const unsigned next = __shfl_down_sync(~0u, bits, 4);

    if (at.slot >= 0) {
        unsigned char *rec = c.pool + record_offset<D>(c, at.slot, at.head);
        reinterpret_cast<unsigned *>(rec + (at.which ? D / 2 : 0))[at.w] = at.which ? vw : kw;
        if (at.w % 8 == 0)
            reinterpret_cast<unsigned *>(rec + D + (at.which ? D / 16 : 0))[at.w / 8] = bits | next << 16;
        if (record_bytes(D) > data_bytes(D) && at.w * 4 < record_bytes(D) - data_bytes(D) && at.which)
            reinterpret_cast<unsigned *>(rec + data_bytes(D))[at.w] = 0;
    }
}

// Codes n and n + 4 of a word, as floats: (code | 1024 in fp16) - 1032 is exact.
__device__ __forceinline__ float2 two_codes(unsigned word, int n)
{
    const unsigned x = (word >> (4 * n) & 0x000f000fu) | 0x64006400u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6408)));
    return __half22float2(h);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(Cache c, Divider by_heads, const int32_t *__restrict__ seq,
            const int32_t *__restrict__ pos, int tokens, T *__restrict__ k, T *__restrict__ v)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);
    const Place<D> at(c, by_heads, seq, pos, tokens);
    unsigned stored = 0x88888888u;
    float scale = 0.f;
    if (at.slot >= 0) {
        const unsigned char *rec = c.pool + record_offset<D>(c, at.slot, at.head);
        stored = reinterpret_cast<const unsigned *>(rec + (at.which ? D / 2 : 0))[at.w];
        scale = __half2float(
            reinterpret_cast<const __half *>(rec + D + (at.which ? D / 16 : 0))[at.w / 4]);
    }
    const unsigned kw = __shfl_sync(~0u, stored, first + key_place<D>(at.w));
    // value: channels 8 w .. 8 w + 7 of the stretch are pieces 2 w and 2 w + 1,
    // (g, i) and (g + 1, i) with i = w / 4, g = 2 (w % 4)
    const int local = at.w & (4 * n - 1), i = local / 4, g = 2 * (local % 4);
    const int base = first + (at.w & ~(4 * n - 1));
    const unsigned lo = __shfl_sync(~0u, stored, base + (n * g + i) / 2);
    const unsigned hi = __shfl_sync(~0u, stored, base + (n * g + n + i) / 2);
    const unsigned vw = __byte_perm(lo, hi, i & 1 ? 0x7632 : 0x5410);
    if (!at.in)
        return;
    const unsigned word = at.which ? vw : kw;
    Eight<T> e;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 f = two_codes(word, j);
        from_float(e.x[j], f.x * scale);
        from_float(e.x[j + 4], f.y * scale);
    }
    T *dst = (at.which ? v : k) + ((long long)at.token * c.kv_heads + at.head) * D;
    *reinterpret_cast<Eight<T> *>(dst + at.w * 8) = e;
}

long long blocks_for(const Cache &c, int d, long long tokens)
{
    const long long rows = tokens * c.kv_heads * 2, each = kThreads / (d / 8);
    return (rows + each - 1) / each;
}

template <typename T, int D>
cudaError_t append_one(const Cache &c, const int32_t *seq, const int32_t *pos, long long tokens,
                       const void *k, const int64_t *ks, const void *v, const int64_t *vs,
                       cudaStream_t stream)
{
    // 16-byte loads where every vector starts on 16 bytes (8 channels of fp32
    // are two of them)
    bool vec = ((uintptr_t)k | (uintptr_t)v) % 16 == 0;
    for (int j = 0; j < 2; ++j)
        vec = vec && ks[j] * (long long)sizeof(T) % 16 == 0 && vs[j] * (long long)sizeof(T) % 16 == 0;
    const unsigned grid = (unsigned)blocks_for(c, D, tokens);
    Divider by_heads;
    by_heads.set(c.kv_heads);
    auto fn = vec ? append_kernel<T, D, true> : append_kernel<T, D, false>;
    fn<<<grid, kThreads, 0, stream>>>(c, by_heads, seq, pos, (int)tokens, (const T *)k, ks[0], ks[1],
                                      (const T *)v, vs[0], vs[1]);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read_one(const Cache &c, const int32_t *seq, const int32_t *pos, long long tokens,
                     void *k, void *v, cudaStream_t stream)
{
    const unsigned grid = (unsigned)blocks_for(c, D, tokens);
    Divider by_heads;
    by_heads.set(c.kv_heads);
    read_kernel<T, D><<<grid, kThreads, 0, stream>>>(c, by_heads, seq, pos, (int)tokens, (T *)k, (T *)v);
    return cudaGetLastError();
}

template <typename T>
cudaError_t append_dim(const Cache &c, int d, const int32_t *seq, const int32_t *pos,
                       long long tokens, const void *k, const int64_t *ks, const void *v,
                       const int64_t *vs, cudaStream_t stream)
{
    return d == 64    ? append_one<T, 64>(c, seq, pos, tokens, k, ks, v, vs, stream)
           : d == 128 ? append_one<T, 128>(c, seq, pos, tokens, k, ks, v, vs, stream)
                      : append_one<T, 256>(c, seq, pos, tokens, k, ks, v, vs, stream);
}

template <typename T>
cudaError_t read_dim(const Cache &c, int d, const int32_t *seq, const int32_t *pos,
                     long long tokens, void *k, void *v, cudaStream_t stream)
{
    return d == 64    ? read_one<T, 64>(c, seq, pos, tokens, k, v, stream)
           : d == 128 ? read_one<T, 128>(c, seq, pos, tokens, k, v, stream)
                      : read_one<T, 256>(c, seq, pos, tokens, k, v, stream);
}

}  // namespace

bool store_fits(const Cache &c, long long tokens)
{
    // (token, head) rows are numbered below 2^31, those of the last CTA too
    return tokens < 1LL << 31 && tokens * c.kv_heads < (1LL << 31) - kThreads;
}

cudaError_t launch_append(const Cache &c, int head_dim, int dtype, const int32_t *seq,
                          const int32_t *pos, long long tokens, const void *k, const int64_t *ks,
                          const void *v, const int64_t *vs, cudaStream_t stream)
{
    return dtype == DS_FP32
               ? append_dim<float>(c, head_dim, seq, pos, tokens, k, ks, v, vs, stream)
           : dtype == DS_BF16
               ? append_dim<__nv_bfloat16>(c, head_dim, seq, pos, tokens, k, ks, v, vs, stream)
               : append_dim<__half>(c, head_dim, seq, pos, tokens, k, ks, v, vs, stream);
}

cudaError_t launch_read(const Cache &c, int head_dim, int dtype, const int32_t *seq,
                        const int32_t *pos, long long tokens, void *k, void *v,
                        cudaStream_t stream)
{
    return dtype == DS_FP32   ? read_dim<float>(c, head_dim, seq, pos, tokens, k, v, stream)
           : dtype == DS_BF16 ? read_dim<__nv_bfloat16>(c, head_dim, seq, pos, tokens, k, v, stream)
                              : read_dim<__half>(c, head_dim, seq, pos, tokens, k, v, stream);
}

}  // namespace kv4
}  // namespace ds
