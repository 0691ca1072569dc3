// ds_kv4_chunk_256.cu -- attention of chunks, head dimension 256.
#include "ds_kv4_chunk.cuh"

namespace ds {
namespace kv4 {

cudaError_t launch_chunk_256(const chunk::Args &p, int dev, int ctas, cudaStream_t stream)
{
    return chunk::launch_chunk_dim<256>(p, dev, ctas, stream);
}

}  // namespace kv4
}  // namespace ds
