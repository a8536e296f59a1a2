// launch_chain.h -- kernels of one call that depend on one another, launched so
// that a kernel's start can overlap the end of the one before (programmatic
// dependent launch; `early`): its CTAs take the SMs that fall free, set themselves
// up and wait in grid_wait() until the kernel before has ended and its writes are
// visible.  Linear attention backward over six ragged sequences of 572 tokens,
// ten kernels: 126 -> 100 us; over one of 8,192: 670 -> 655 us.
//
// The rules that make this safe:
//  - the call's first kernel is launched as usual, behind all earlier work of the stream;
//  - every CTA of every kernel runs grid_wait() before it touches global memory
//    that an earlier kernel of the call reads or writes, and before it ends, so
//    that a kernel that has ended implies that all before it have;
//  - grid_next() comes after grid_wait() in every kernel but the first: at most one kernel is set up ahead.
#pragma once

#include <cuda_runtime.h>

namespace gdn {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

struct Chain {
    cudaStream_t stream;
    bool begun = false;

    template <typename... Params, typename... Args>
    cudaError_t launch(bool early, void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                       const Args&... args) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr.val.programmaticStreamSerializationAllowed = 1;
        cudaLaunchConfig_t config{};
        config.gridDim = grid;
        config.blockDim = dim3(threads);
        config.dynamicSmemBytes = smem;
        config.stream = stream;
        config.attrs = &attr;
        config.numAttrs = begun && early ? 1 : 0;
        begun = true;
        return cudaLaunchKernelEx(&config, kernel, args...);
    }
};

}  // namespace gdn
