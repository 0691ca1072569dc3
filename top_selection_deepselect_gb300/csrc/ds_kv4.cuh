// ds_kv4.cuh -- the 4-bit cache as the kernels see it: record layout, page
// lookup, conversions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_topk.h"

namespace ds {
namespace kv4 {

constexpr int kGroup = 32;  // channels that share a scale

__host__ __device__ constexpr int data_bytes(int d) { return d + 4 * (d / kGroup); }
__host__ __device__ constexpr int record_bytes(int d) { return (data_bytes(d) + 15) / 16 * 16; }

// Quotient by a fixed divisor of numbers below 2^31: n d' / 2^shift with
// d' = 2^shift / d rounded up, shift = 31 + ceil(log2 d), which is exact there.
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

struct Cache {
    unsigned char *pool;
    long long page_stride;
    const int32_t *table;
    long long table_stride;
    int n_pages, page_size, kv_heads, max_seqs, max_pages;
    Divider by_page;
};

// Loads below are plain ones on purpose: a kernel that starts while the previous
// one drains may not read what that one writes through the read-only path, whose
// loads may also be moved before the wait.

// Page and offset in it of position `pos` of sequence `seq`; page -1 where the
// sequence, the position or the page is out of range.
struct Slot {
    int page, offset;
};

__device__ __forceinline__ Slot token_slot(const Cache &c, int seq, int pos)
{
    if ((unsigned)seq >= (unsigned)c.max_seqs || pos < 0)
        return {-1, 0};
    const int col = c.by_page(pos);
    if (col >= c.max_pages)
        return {-1, 0};
    const int page = c.table[seq * c.table_stride + col];
    return {(unsigned)page < (unsigned)c.n_pages ? page : -1, pos - col * c.page_size};
}

// Byte offset of the record of (slot, head) in the pool: 64 bits, a pool may
// be hundreds of gigabytes.
template <int D>
__device__ __forceinline__ long long record_offset(const Cache &c, const Slot &s, int head)
{
    return s.page * c.page_stride + ((long long)head * c.page_size + s.offset) * record_bytes(D);
}

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ void from_float(float &y, float x) { y = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16 &y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_float(__half &y, float x) { y = __float2half_rn(x); }

}  // namespace kv4
}  // namespace ds
