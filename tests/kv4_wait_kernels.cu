// Test kernel for the wait of the 4-bit cache's attention on its arrival
// barriers (test infrastructure only).  Warp 0 waits, its lane 0 and the others
// starting at times of their own; warp 1 arrives at a time, or never.  All times
// are waited for by the clock, with a limit on the number of looks at it.
#include "ds_kv4_attention.cuh"

using namespace ds::kv4;

__device__ void until(long long start, long long ns)
{
    for (int i = 0; i < 100000000 && nanoseconds() - start < ns; ++i) {
    }
}

__global__ void k_wait(long long lane0, long long others, long long arrival, long long patience, int *came)
{
    __shared__ alignas(8) unsigned long long barrier;
    const uint32_t bar = shared_address(&barrier);
    if (threadIdx.x == 0)
        barrier_init(bar);
    __syncthreads();
    const long long start = nanoseconds();
    if (threadIdx.x < 32) {
        bool late = false;
        if (threadIdx.x == 0) {
            until(start, lane0);
            barrier_wait(bar, 0, late, patience);
        } else {
            until(start, others);
            barrier_wait(bar, 0, late, patience);
        }
        came[threadIdx.x] = !__any_sync(~0u, late);
    } else if (threadIdx.x == 32 && arrival >= 0) {
        until(start, arrival);
        barrier_expect(bar, 0);
    }
    __syncthreads();
}

extern "C" int wait_of(long long lane0, long long others, long long arrival, long long patience, int *came)
{
    k_wait<<<1, 64>>>(lane0, others, arrival, patience, came);
    return (int)cudaDeviceSynchronize();
}
