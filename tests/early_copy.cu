// A copy that lets the next kernel in its stream start at once and writes late: what a
// producer under programmatic dependent launch may do.
#include <cuda_runtime.h>
#include <stdint.h>

__device__ static unsigned long long now_ns() {
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__global__ void early_copy_kernel(uint32_t *dst, const uint32_t *src, long long words, unsigned long long ns) {
    asm volatile("griddepcontrol.launch_dependents;");
    const unsigned long long t0 = now_ns();
    for (int i = 0; i < (1 << 18) && now_ns() - t0 < ns; ++i) {
    }
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < words; i += (long long)gridDim.x * blockDim.x) dst[i] = src[i];
}

// Copies `bytes` (a multiple of 4) after `ns` nanoseconds.
extern "C" int early_copy(void *dst, const void *src, long long bytes, unsigned long long ns, void *stream) {
    early_copy_kernel<<<32, 256, 0, (cudaStream_t)stream>>>((uint32_t *)dst, (const uint32_t *)src, bytes / 4, ns);
    return (int)cudaGetLastError();
}
