// A grid that lets the next one in its stream start at once (programmatic dependent launch) and writes only
// after a while, for the tests of calls whose inputs such a grid makes.
#include <cuda_runtime.h>
#include <stdint.h>

__global__ void late_copy_kernel(const uint4 *from, uint4 *to, size_t n, uint64_t ns) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < 1000000; ++i) {  // ends by itself, whatever the timer does
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 >= ns) break;
    }
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x)
        to[i] = from[i];
}

extern "C" __attribute__((visibility("default"))) int late_copy(const void *from, void *to, size_t bytes,
                                                                  unsigned long long ns, int grid, void *stream) {
    late_copy_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4 *>(from), static_cast<uint4 *>(to), bytes / 16, ns);
    return (int)cudaGetLastError();
}
