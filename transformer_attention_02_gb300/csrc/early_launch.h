// Programmatic dependent launch, for the kernels of a decode step and the
// windowed attention.
#pragma once

#include <cuda_runtime.h>

namespace attn {

// Launches a kernel that may become resident while the kernel before it in the
// stream drains (programmatic dependent launch). Such a kernel begins with
// wait_for_inputs(): nothing of it touches memory before everything earlier in
// the stream has finished and is visible. Saves most of the launch latency
// between the steps of a decode loop.
// Visible to ordinary loads, that is. The non-coherent ones (__ldg) are for data
// that nothing writes as long as the kernel lives, and it lives while the kernel
// before it still writes: they read rotation tables only, which no kernel that lets
// its successor start early makes. Data of the stream is read by plain loads, or, where
// it is read once or a neighbour's line may be in L1, by __ldcg from L2.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream,
                         Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_inputs() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel of the stream may become resident from here on.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
#endif

}  // namespace attn
