// stream_order.cuh -- kernels that are set up while the one before them on the stream still runs. Such a
// kernel calls wait_for_stream() in every thread, behind which all that was before it on the stream is done.
//
// Before the wait it may touch only what nothing in flight writes. A kernel that a call launches first cannot
// know what runs before it, so it reads and writes nothing before the wait. A later one of the same call
// may read what was there before the call, if every block of the launch before it lets it start
// (griddepcontrol.launch_dependents) behind its own wait, and that launch does not write what is read: all that was
// before the call is then done. The plan's second launch does so (pages.cu). Nothing is written before the wait
// but bits that are OR-ed into the status word.
//
// Between small kernels this saves about a microsecond each.
#pragma once

#include <cuda_runtime.h>

namespace stq {

#ifdef __CUDACC__
__device__ __forceinline__ void wait_for_stream() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
#endif

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t s, const A &...args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace stq
