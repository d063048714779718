// cg_launch.cuh -- programmatic launch: a kernel that may start while the one
// before it in the stream still runs (sm_103a).
#pragma once

#include <cuda_runtime.h>

namespace cg {

// On the device: the next kernel of the stream may start now; and wait for
// the kernel before this one to be complete and its writes visible.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// With `early` the kernel may start before the one ahead of it is done; it
// then calls wait_for_previous before it touches that one's results.
template <class... P, class... A>
cudaError_t launch_next(void (*k)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, bool early,
                        const A &...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &at;
    c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, k, args...);
}

}  // namespace cg
