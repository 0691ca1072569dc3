// ds_kv4_store.cu -- append to and read from the 4-bit cache.
//
// One lane holds eight channels of one token's key or value (16 bytes of a
// 16-bit type), so a vector of D channels takes D/8 neighbouring lanes and a
// group of 32 channels four of them: the group's largest magnitude is two
// shuffles away, and the reordering inside the record is a shuffle too, so that
// codes leave and arrive as whole words.  Both kernels move each byte once.
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

// What a lane works on: token, head, key or value, and word w of the vector.
template <int D>
struct Place {
    long long token;
    int head, which, w, slot;
    bool in;
    __device__ Place(const Cache &c, const int32_t *seq, const int32_t *pos, long long tokens)
    {
        const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
        w = (int)(i % (D / 8));
        const long long r = i / (D / 8);
        which = (int)(r & 1);
        head = (int)((r >> 1) % c.kv_heads);
        token = (r >> 1) / c.kv_heads;
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

template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(kThreads)
append_kernel(Cache c, const int32_t *__restrict__ seq, const int32_t *__restrict__ pos,
              long long tokens, const T *__restrict__ k, long long k_token, long long k_head,
              const T *__restrict__ v, long long v_token, long long v_head)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    const Place<D> at(c, seq, pos, tokens);
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);

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

    // scale of the group; a NaN or an infinity poisons it
    float most = 0.f;
    int bad = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float a = fabsf(x[j]);
        bad |= !(a <= 3.402823466e38f);
        most = fmaxf(most, a);
    }
    most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
    most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
    bad |= __shfl_xor_sync(~0u, bad, 1);
    bad |= __shfl_xor_sync(~0u, bad, 2);
    __half scale = __float2half_rn(most / 7.f);
    if (__hisinf(scale))
        scale = __ushort_as_half(0x7bff);
    const float step = __half2float(scale);
    unsigned word = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float q = step > 0.f && !bad ? rintf(x[j] / step) : 0.f;
        q = fminf(fmaxf(q, -7.f), 7.f);
        word |= (unsigned)((int)q + 8) << (4 * j);
    }
    unsigned bits = __half_as_ushort(scale);
    if (bad)
        bits = 0x7fffu;

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

    if (at.slot < 0)
        return;
    unsigned char *rec = c.pool + record_offset<D>(c, at.slot, at.head);
    reinterpret_cast<unsigned *>(rec + (at.which ? D / 2 : 0))[at.w] = at.which ? vw : kw;
    if (at.w % 8 == 0)
        reinterpret_cast<unsigned *>(rec + D + (at.which ? D / 16 : 0))[at.w / 8] = bits | next << 16;
    if (record_bytes(D) > data_bytes(D) && at.w * 4 < record_bytes(D) - data_bytes(D) && at.which)
        reinterpret_cast<unsigned *>(rec + data_bytes(D))[at.w] = 0;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(Cache c, const int32_t *__restrict__ seq, const int32_t *__restrict__ pos,
            long long tokens, T *__restrict__ k, T *__restrict__ v)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    const Place<D> at(c, seq, pos, tokens);
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);
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
    for (int j = 0; j < 8; ++j)
        from_float(e.x[j], (float)((int)(word >> (4 * j) & 15) - 8) * scale);
    T *dst = (at.which ? v : k) + (at.token * c.kv_heads + at.head) * D;
    *reinterpret_cast<Eight<T> *>(dst + at.w * 8) = e;
}

long long blocks_for(const Cache &c, int d, long long tokens)
{
    return (tokens * c.kv_heads * 2 * (d / 8) + kThreads - 1) / kThreads;
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
    auto fn = vec ? append_kernel<T, D, true> : append_kernel<T, D, false>;
    fn<<<grid, kThreads, 0, stream>>>(c, seq, pos, tokens, (const T *)k, ks[0], ks[1],
                                      (const T *)v, vs[0], vs[1]);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t read_one(const Cache &c, const int32_t *seq, const int32_t *pos, long long tokens,
                     void *k, void *v, cudaStream_t stream)
{
    const unsigned grid = (unsigned)blocks_for(c, D, tokens);
    read_kernel<T, D><<<grid, kThreads, 0, stream>>>(c, seq, pos, tokens, (T *)k, (T *)v);
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

long long store_blocks(const Cache &c, int head_dim, long long tokens)
{
    return blocks_for(c, head_dim, tokens);
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
