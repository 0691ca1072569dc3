// ds_kv4_launch.h -- launchers behind the entry points of ds_kv4.h: arguments
// are checked by the callers, the launch's status comes back.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace ds {
namespace kv4 {

struct Cache;

// Whether append and read can number the rows of so many tokens.
bool store_fits(const Cache &c, long long tokens);
cudaError_t launch_append(const Cache &c, int head_dim, int dtype, const int32_t *seq,
                          const int32_t *pos, long long tokens, const void *k, const int64_t *ks,
                          const void *v, const int64_t *vs, cudaStream_t stream);
cudaError_t launch_read(const Cache &c, int head_dim, int dtype, const int32_t *seq,
                        const int32_t *pos, long long tokens, void *k, void *v,
                        cudaStream_t stream);

// One call of attention.
struct Attend {
    const int32_t *lengths, *seqs, *indices;
    const void *q;
    long long q_batch, q_query, q_head;  // strides in elements
    void *out;
    float *lse;
    float *partial;  // workspace
    float scale;
    int batch, queries, heads, k;
    int bf16;        // 1: q and out are bf16, 0: fp16
};

// Workspace that a call of these sizes (batch, queries, heads, k) needs.
size_t attention_workspace(const Cache &c, int head_dim, const Attend &a, int sms);
cudaError_t launch_attention(const Cache &c, int head_dim, const Attend &a, int dev, int sms,
                             cudaStream_t stream);

}  // namespace kv4
}  // namespace ds
