// ds_kv4_attention.cu -- attention over the 4-bit cache: choice of the head
// dimension's instantiation and the workspace's size.
#include "ds_kv4_attention.cuh"

namespace ds {
namespace kv4 {

cudaError_t launch_attention_64(const Cache &c, const Attend &a, int dev, int sms, cudaStream_t stream);
cudaError_t launch_attention_128(const Cache &c, const Attend &a, int dev, int sms, cudaStream_t stream);
cudaError_t launch_attention_256(const Cache &c, const Attend &a, int dev, int sms, cudaStream_t stream);

size_t attention_workspace(const Cache &c, int head_dim, const Attend &a, int sms)
{
    return head_dim == 64    ? workspace_dim<64>(c, a, sms)
           : head_dim == 128 ? workspace_dim<128>(c, a, sms) : workspace_dim<256>(c, a, sms);
}

cudaError_t launch_attention(const Cache &c, int head_dim, const Attend &a, int dev, int sms,
                             cudaStream_t stream)
{
    return head_dim == 64    ? launch_attention_64(c, a, dev, sms, stream)
           : head_dim == 128 ? launch_attention_128(c, a, dev, sms, stream)
                             : launch_attention_256(c, a, dev, sms, stream);
}

}  // namespace kv4
}  // namespace ds
