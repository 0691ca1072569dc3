// ds_kv4_attention.cu -- attention over the 4-bit cache.
#include "ds_kv4.cuh"
#include "ds_kv4_launch.h"

namespace ds {
namespace kv4 {
namespace {

// One warp per (sequence, query, head): a lane holds the channels of one word
// of the key and, for the value, the channels of the same word.
template <int D, typename T>
__global__ void attention_kernel(Cache c, Attend a)
{
    constexpr int n = (D < 128 ? D : 128) / kGroup;
    const int lane = threadIdx.x & 31, w = lane;
    const long long row = (long long)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
    if (row >= (long long)a.batch * a.queries * a.heads)
        return;
    const int h = (int)(row % a.heads);
    const int j = (int)(row / a.heads % a.queries);
    const int b = (int)(row / a.heads / a.queries);
    const int head = h / (a.heads / c.kv_heads);
    const int seq = a.seqs ? a.seqs[b] : b;
    int len = (unsigned)seq < (unsigned)c.max_seqs ? a.lengths[seq] : 0;
    const long long room = (long long)c.max_pages * c.page_size;
    len = len < 0 ? 0 : len > room ? (int)room : len;
    const int limit = len - a.queries + 1 + j;
    const int count = a.indices ? a.k : limit;
    const int32_t *list = a.indices ? a.indices + ((long long)b * a.queries + j) * a.k : nullptr;
    const T *q = (const T *)a.q + b * a.q_batch + j * a.q_query + h * a.q_head;
    float x[8], o[8], m = -INFINITY, l = 0.f;
    for (int e = 0; e < 8; ++e) {
        x[e] = w < D / 8 ? to_float(q[w * 8 + e]) : 0.f;
        o[e] = 0.f;
    }
    const int part = w / (4 * n), local = w % (4 * n);
    const int kplace = part * 4 * n + n * (local % 4) + local / 4;
    const int i = local / 4, g = 2 * (local % 4);
    const int vplace = part * 8 * n + n * g + i;
    for (int t = 0; t < count; ++t) {
        const int pos = list ? list[t] : t;
        if (pos < 0 || pos >= limit)
            continue;
        const int slot = token_slot(c, seq, pos);
        if (slot < 0)
            continue;
        const unsigned char *rec = c.pool + record_offset<D>(c, slot, head);
        float s = 0.f, vs = 0.f;
        unsigned vw = 0;
        if (w < D / 8) {
            const unsigned kw = reinterpret_cast<const unsigned *>(rec)[kplace];
            for (int e = 0; e < 8; ++e)
                s += x[e] * (float)((int)(kw >> (4 * e) & 15) - 8);
            s *= __half2float(reinterpret_cast<const __half *>(rec + D)[w / 4]);
            const unsigned short *vh = reinterpret_cast<const unsigned short *>(rec + D / 2);
            vw = vh[vplace] | (unsigned)vh[vplace + n] << 16;
            vs = __half2float(reinterpret_cast<const __half *>(rec + D + D / 16)[w / 4]);
        }
        for (int step = 16; step; step /= 2)
            s += __shfl_xor_sync(~0u, s, step);
        s *= a.scale;
        const float top = fmaxf(m, s), old = m == top ? 1.f : expf(m - top), p = expf(s - top);
        m = top;
        l = l * old + p;
        for (int e = 0; e < 8; ++e)
            o[e] = o[e] * old + p * (float)((int)(vw >> (4 * e) & 15) - 8) * vs;
    }
    if (w < D / 8) {
        T *out = (T *)a.out + row * D;
        for (int e = 0; e < 8; ++e)
            from_float(out[w * 8 + e], l == 0.f ? 0.f : o[e] / l);
    }
    if (a.lse && lane == 0)
        a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
}

template <int D>
cudaError_t one(const Cache &c, const Attend &a, cudaStream_t stream)
{
    const long long rows = (long long)a.batch * a.queries * a.heads;
    const unsigned grid = (unsigned)((rows + 3) / 4);
    if (a.bf16)
        attention_kernel<D, __nv_bfloat16><<<grid, 128, 0, stream>>>(c, a);
    else
        attention_kernel<D, __half><<<grid, 128, 0, stream>>>(c, a);
    return cudaGetLastError();
}

}  // namespace

size_t attention_workspace(const Cache &, int, int, int, int, int, int) { return 0; }

cudaError_t launch_attention(const Cache &c, int head_dim, const Attend &a, int,
                             cudaStream_t stream)
{
    return head_dim == 64 ? one<64>(c, a, stream)
           : head_dim == 128 ? one<128>(c, a, stream) : one<256>(c, a, stream);
}

}  // namespace kv4
}  // namespace ds
