// ds_kv4_store.cu -- append to and read from the 4-bit cache.
//
// One lane holds eight channels of one token's key and the same of its value (16
// bytes each of a 16-bit type), so a vector of D channels takes D/8 neighbouring
// lanes and a group of 32 channels four of them: the group's largest magnitude
// is two shuffles away (one for both the key's and the value's, whose scales are
// worked out in turn by neighbouring lanes), and the reordering inside the record is a shuffle too,
// so that codes leave and arrive as whole words.  Both kernels move each byte
// once and are bound by the bytes only while a lane's eight channels cost few
// instructions: magnitudes are compared as bits, quotients and integers come
// from multiply-adds, and a token's place is looked up once for several heads
// where there are tokens enough.
#include "ds_device.cuh"
#include "ds_host.h"
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

// What a lane works on: rows of D/8 lanes are (token, run of `each` heads), the
// last fastest.
template <int D>
struct Place {
    int token, head, w;
    bool in;
    Slot slot;
    __device__ __forceinline__ Place(const Cache &c, const Divider &by_runs, int each, int runs,
                                     const int32_t *seq, const int32_t *pos,
                                     int tokens)
    {
        w = threadIdx.x % (D / 8);
        const int row = blockIdx.x * (kThreads / (D / 8)) + threadIdx.x / (D / 8);   // below 2^31
        token = by_runs(row);
        head = (row - token * runs) * each;
        in = token < tokens;
        slot = in ? token_slot(c, seq[token], pos[token]) : Slot{-1, 0};
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

template <typename T, bool kVec>
__device__ __forceinline__ Eight<T> load_eight(const T *src)
{
    Eight<T> e;
    if constexpr (kVec) {
        e = *reinterpret_cast<const Eight<T> *>(src);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            e.x[j] = src[j];
    }
    return e;
}

// Largest magnitude of a lane's eight channels, as the bits of a float: the bits
// of magnitudes are in their order, those that are not finite above all others,
// in 16-bit types two at a time.
__device__ __forceinline__ unsigned largest(const Eight<float> &e)
{
    unsigned most = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        most = max(most, __float_as_uint(e.x[j]) & 0x7fffffffu);
    return most;
}

template <typename T>
__device__ __forceinline__ unsigned largest(const Eight<T> &e)
{
    const unsigned *w = reinterpret_cast<const unsigned *>(&e);
    unsigned most = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < 4; ++j)
        most = __vmaxu2(most, w[j] & 0x7fff7fffu);
    const unsigned short top = (unsigned short)max(most & 0xffffu, most >> 16);
    return __float_as_uint(to_float(*reinterpret_cast<const T *>(&top)));
}

// Scale of a group: its bits, what codes are made with (0 where the codes are
// all 8) and the nearest float to 1 / step.
struct Scale {
    unsigned bits;
    float inv;
};

__device__ __forceinline__ float step_of(unsigned bits)
{
    return __half2float(__ushort_as_half((unsigned short)bits));
}

__device__ __forceinline__ Scale scale_of(unsigned most)
{
    __half scale = __float2half_rn(__uint_as_float(most) * (1.f / 7.f));
    if (__hisinf(scale))
        scale = __ushort_as_half(0x7bff);
    const bool bad = most >= 0x7f800000u;      // a NaN or an infinity poisons the group
    return {bad ? 0x7fffu : __half_as_ushort(scale), __frcp_rn(__half2float(scale))};
}

// Bits of the floats round(round(x[i] f + a) + b), a pair in one instruction each.
__device__ __forceinline__ void multiply_add_add(float x0, float x1, float f, float a, float b,
                                                 unsigned *y0, unsigned *y1)
{
    asm("{\n\t"
        ".reg .b64 x, f, a, b;\n\t"
        "mov.b64 x, {%2, %3};\n\t"
        "mov.b64 f, {%4, %4};\n\t"
        "mov.b64 a, {%5, %5};\n\t"
        "mov.b64 b, {%6, %6};\n\t"
        "fma.rn.f32x2 x, x, f, a;\n\t"
        "add.rn.f32x2 x, x, b;\n\t"
        "mov.b64 {%0, %1}, x;\n\t"
        "}"
        : "=r"(*y0), "=r"(*y1)
        : "f"(x0), "f"(x1), "f"(f), "f"(a), "f"(b));
}

// Codes of the lane's eight channels.  wide: some quotient of the warp's may be
// beyond 7.
template <typename T>
__device__ __forceinline__ unsigned encode(const Eight<T> &e, const Scale &s, bool wide)
{
    // the float q + 12582920 (1.5 2^23 + 8) holds rint(q) + 8 in its low bits,
    // above a constant that the sum takes away once for all eight
    unsigned word = 0;
    if (sizeof(T) == 2 && !wide) {
        // q to the nearest multiple of 2^-13 first, by adding 1536.  With 11
        // significant bits in x and in the scale a quotient that is no tie is
        // 2^-12.2 away from one at least, so that it stays on its side, and a
        // tie, whose product may be a little off, is met exactly: the integer
        // is the rounded quotient's, and the correction is saved.
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            unsigned lo, hi;
            multiply_add_add(to_float(e.x[j]), to_float(e.x[j + 1]), s.inv, 1536.f, 12581384.f, &lo, &hi);
            word += (lo << (4 * j)) + (hi << (4 * j + 4));
        }
    } else {
        const float step = step_of(s.bits);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float q = quotient(to_float(e.x[j]), step, s.inv);
            if (wide)
                q = fminf(fmaxf(q, -7.f), 7.f);
            word += __float_as_uint(q + 12582920.f) << (4 * j);
        }
    }
    return s.bits == 0 || s.bits == 0x7fffu ? 0x88888888u : word - 0x3f400000u;
}

// 31.9 us for 28693 tokens of 8 heads of 128 in bf16 (150 MB, 4.7 TB/s), 43.9 in
// fp32 (268 MB, 6.1 TB/s).  16-bit types lie between two bounds: some 220
// instructions for a lane's 16 channels keep issue 69 % and the ALU 67 % busy, and
// waits for loads are the largest stall.  A pair a multiply-add 32.8 -> 31.9, scales shared out and no
// correction 35.1 -> 32.8; six CTAs an SM (five 33.4; seven and eight spill, 33.1);
// the next head's loads ahead of this one's codes, or two heads at once, are slower
// (39.9, 34.5).
template <typename T, int D, bool kVec>
__global__ void __launch_bounds__(kThreads, 6)
append_kernel(Cache c, Divider by_runs, int each, int runs, const int32_t *seq,
              const int32_t *pos, int tokens, const T *k, long long k_token,
              long long k_head, const T *v, long long v_token, long long v_head)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    dependent_grid_wait();
    allow_dependent_grid();
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);
    const Place<D> at(c, by_runs, each, runs, seq, pos, tokens);
    const bool there = at.slot.page >= 0;
    // a lane whose token is not there reads the first one's, and writes nothing
    const int token = there ? at.token : 0, head = there ? at.head : 0;
    k += token * k_token + head * k_head + at.w * 8;
    v += token * v_token + head * v_head + at.w * 8;
    unsigned char *rec = c.pool + (there ? record_offset<D>(c, at.slot, at.head) : 0);

    // stored order: source lanes.  Value word p holds pieces (g, i) and (g, i + 1),
    // n g + i = 2 p within the stretch; piece (g, i) is half g & 1 of word 4 i + g / 2
    const int local = at.w & (4 * n - 1), g = 2 * local / n, i = 2 * local % n;
    const int from_k = first + key_source<D>(at.w);
    const int from_v = first + (at.w & ~(4 * n - 1)) + g / 2 + 4 * i;
    const unsigned pick = g & 1 ? 0x7632 : 0x5410;
    // the word of scales that this lane writes, if any: key scales by the first
    // lane of two groups, value scales by the second
    const bool scales = at.w % 4 == 0, right = lane & 1;

#pragma unroll 1
    for (int h = 0; h < each; ++h) {
        const Eight<T> x = load_eight<T, kVec>(k), y = load_eight<T, kVec>(v);
        // the group's four lanes: even ones find the key's scale, odd ones the
        // value's, and neighbours exchange them
        const unsigned kmost = largest(x), vmost = largest(y);
        const unsigned given = __shfl_xor_sync(~0u, right ? kmost : vmost, 1);
        unsigned most = max(right ? vmost : kmost, given);
        most = max(most, __shfl_xor_sync(~0u, most, 2));
        const Scale mine = scale_of(most);
        const Scale its = {__shfl_xor_sync(~0u, mine.bits, 1), __shfl_xor_sync(~0u, mine.inv, 1)};
        const Scale ks = right ? its : mine, vs = right ? mine : its;
        // subnormal and largest scales: quotients may be beyond 7 (rare, so a
        // branch)
        const bool wide = __any_sync(~0u, mine.bits < 0x400u || mine.bits >= 0x7bffu);
        const unsigned kbits = ks.bits, vbits = vs.bits;
        const unsigned kc = encode(x, ks, wide), vc = encode(y, vs, wide);
        const unsigned kw = __shfl_sync(~0u, kc, from_k);
        const unsigned lo = __shfl_sync(~0u, vc, from_v), hi = __shfl_sync(~0u, vc, from_v + 4);
        // groups 2 i and 2 i + 1 are four lanes apart: the even one gets both
        // key scales, the odd one both value scales
        const bool odd = at.w & 4;
        const unsigned other = __shfl_xor_sync(~0u, odd ? kbits : vbits, 4);
        const unsigned pair = odd ? other | vbits << 16 : kbits | other << 16;
        if (there) {
            reinterpret_cast<unsigned *>(rec)[at.w] = kw;
            reinterpret_cast<unsigned *>(rec + D / 2)[at.w] = __byte_perm(lo, hi, pick);
            if (scales)
                reinterpret_cast<unsigned *>(rec + D + (odd ? D / 16 : 0))[at.w / 8] = pair;
            if (record_bytes(D) > data_bytes(D) && at.w * 4 < record_bytes(D) - data_bytes(D))
                reinterpret_cast<unsigned *>(rec + data_bytes(D))[at.w] = 0;
        }
        k += there ? k_head : 0;
        v += there ? v_head : 0;
        rec += there ? (long long)c.page_size * record_bytes(D) : 0;
    }
}

// Channels 8 w .. 8 w + 7 of a word of codes: (code | 1024 in fp16) - 1032 is
// exact; nibbles n and n + 4 come out together.
template <typename T>
__device__ __forceinline__ Eight<T> decode(unsigned word, float scale)
{
    Eight<T> e;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const unsigned x = (word >> (4 * j) & 0x000f000fu) | 0x64006400u;
        const float2 f = __half22float2(
            __hsub2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x6408))));
        from_float(e.x[j], f.x * scale);
        from_float(e.x[j + 4], f.y * scale);
    }
    return e;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
read_kernel(Cache c, Divider by_runs, int each, int runs, const int32_t *seq,
            const int32_t *pos, int tokens, T *k, T *v)
{
    constexpr int kWords = D / 8;
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    dependent_grid_wait();
    allow_dependent_grid();
    const int lane = threadIdx.x & 31, first = lane & ~(kWords - 1);
    const Place<D> at(c, by_runs, each, runs, seq, pos, tokens);
    const bool there = at.slot.page >= 0;
    const unsigned char *rec = c.pool + (there ? record_offset<D>(c, at.slot, at.head) : 0);
    const long long to = ((long long)at.token * c.kv_heads + at.head) * D + at.w * 8;
    // value: channels 8 w .. 8 w + 7 of the stretch are pieces 2 w and 2 w + 1,
    // (g, i) and (g + 1, i) with i = w / 4, g = 2 (w % 4)
    const int local = at.w & (4 * n - 1), i = local / 4, g = 2 * (local % 4);
    const int base = first + (at.w & ~(4 * n - 1));
    const int from_k = first + key_place<D>(at.w);
    const int from_v0 = base + (n * g + i) / 2, from_v1 = base + (n * g + n + i) / 2;
    const unsigned pick = i & 1 ? 0x7632 : 0x5410;
#pragma unroll 1
    for (int h = 0; h < each; ++h) {
        unsigned ks = 0x88888888u, vs = 0x88888888u;
        float kscale = 0.f, vscale = 0.f;
        if (there) {
            ks = reinterpret_cast<const unsigned *>(rec)[at.w];
            vs = reinterpret_cast<const unsigned *>(rec + D / 2)[at.w];
            kscale = __half2float(reinterpret_cast<const __half *>(rec + D)[at.w / 4]);
            vscale = __half2float(reinterpret_cast<const __half *>(rec + D + D / 16)[at.w / 4]);
        }
        const unsigned kw = __shfl_sync(~0u, ks, from_k);
        const unsigned lo = __shfl_sync(~0u, vs, from_v0), hi = __shfl_sync(~0u, vs, from_v1);
        if (at.in) {
            *reinterpret_cast<Eight<T> *>(k + to + h * D) = decode<T>(kw, kscale);
            *reinterpret_cast<Eight<T> *>(v + to + h * D) = decode<T>(__byte_perm(lo, hi, pick), vscale);
        }
        rec += there ? (long long)c.page_size * record_bytes(D) : 0;
    }
}

// Launch shape: heads that a lane takes one after another (1, 2 or 4, a divisor
// of kv_heads).  More than one saves looking the token up again, but only where
// the rest still fills the GPU (kFill threads): 28693 tokens of 8 heads of 128
// are appended and read in 61 us with four heads, in 66 us with two and in 80 us
// with one; 64 tokens in 14 us with four and in 10 us with one.
constexpr long long kFill = 1 << 19;

struct Launch {
    int each, runs;
    unsigned grid;
    Divider by_runs;
    Launch(const Cache &c, int d, long long tokens)
    {
        each = 1;
        while (each < 4 && c.kv_heads % (2 * each) == 0 &&
               tokens * (c.kv_heads / (2 * each)) * (d / 8) >= kFill)
            each *= 2;
        runs = c.kv_heads / each;
        const long long rows = tokens * runs, per = kThreads / (d / 8);
        grid = (unsigned)((rows + per - 1) / per);
        by_runs.set(runs);
    }
};

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
    const Launch l(c, D, tokens);
    auto fn = vec ? append_kernel<T, D, true> : append_kernel<T, D, false>;
    return launch_overlapped(fn, l.grid, kThreads, 0, stream, c, l.by_runs, l.each, l.runs, seq, pos,
                             (int)tokens, (const T *)k, ks[0], ks[1], (const T *)v, vs[0], vs[1]);
}

template <typename T, int D>
cudaError_t read_one(const Cache &c, const int32_t *seq, const int32_t *pos, long long tokens,
                     void *k, void *v, cudaStream_t stream)
{
    const Launch l(c, D, tokens);
    return launch_overlapped(read_kernel<T, D>, l.grid, kThreads, 0, stream, c, l.by_runs, l.each, l.runs,
                             seq, pos, (int)tokens, (T *)k, (T *)v);
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
