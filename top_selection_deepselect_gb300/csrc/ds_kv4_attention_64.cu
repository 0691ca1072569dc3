// Attention over the 4-bit cache, head dimension 64.
#include "ds_kv4_attention.cuh"

namespace ds {
namespace kv4 {

cudaError_t launch_attention_64(const Cache &c, const Attend &a, int dev, int sms, cudaStream_t stream)
{
    return launch_dim<64>(c, a, dev, sms, stream);
}

}  // namespace kv4
}  // namespace ds
