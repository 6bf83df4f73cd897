// A kernel of other code that lets its successor start between its wait for its own
// predecessor and its stores: dst = src, `hold_ns` later.
#include <cstdint>
#include <cuda_runtime.h>

__global__ void early_producer(uint4 *dst, const uint4 *src, int n, uint64_t hold_ns) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    uint64_t t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    for (int i = 0; i < 1000000; ++i) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (t - t0 >= hold_ns) break;
    }
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = src[i];
}

// n: 16-byte words.
extern "C" int launch_early_producer(void *dst, const void *src, int n, uint64_t hold_ns, void *stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, early_producer, static_cast<uint4 *>(dst), static_cast<const uint4 *>(src), n, hold_ns);
}
