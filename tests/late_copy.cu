// A producer for the tests of early launches: lets the next kernel in at once, then waits,
// and only then writes what that kernel reads.
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void late_copy_kernel(const uint4 *src, uint4 *dst, long long n, unsigned long long ns)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < (1 << 20); ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 >= ns)
            break;
    }
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x)
        dst[i] = src[i];
}

extern "C" int late_copy(const void *src, void *dst, long long vectors, unsigned long long ns, void *stream)
{
    late_copy_kernel<<<32, 256, 0, static_cast<cudaStream_t>(stream)>>>(static_cast<const uint4 *>(src),
                                                                        static_cast<uint4 *>(dst), vectors, ns);
    return static_cast<int>(cudaGetLastError());
}
