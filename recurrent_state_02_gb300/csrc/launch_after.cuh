// launch_after.cuh -- a kernel whose CTAs may start while the one before it in the stream ends (programmatic dependent launch):
// its launch and its set-up are then out of the way when that one's results are there.
#pragma once

#include <cuda_runtime.h>

namespace la {
namespace {

// In the earlier kernel: the next one may be placed once every CTA has been here (or has ended).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// In the later one, before it reads what the earlier kernel writes or writes what that one reads or writes: it has ended here, and what it
// wrote is visible.  (What neither touches may come before: inputs that were ready when the earlier one was launched in the ordinary way,
// and memory of one's own.)  An earlier kernel that has waited here itself has seen the one before it end.  Nothing after an ordinary launch.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute early = {};
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace
}  // namespace la
