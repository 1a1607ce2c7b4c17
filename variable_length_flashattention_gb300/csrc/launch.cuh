// launch.cuh -- launches that may start while the kernel before them in the
// stream is still running (programmatic stream serialisation).
//
// What orders them.  griddepcontrol.wait waits for the one grid ahead: for it to
// end and for its writes to be visible.  The grids ahead of that one are done only
// if it waited for them itself, so every kernel launched this way waits before it
// ends, also where it has nothing to do or leaves early (the backward's dQ kernel
// and the paged decode step, which start ahead of their wait, among them).  A
// kernel that never says launch_dependents lets the next one start at its end,
// with its writes visible: what may be read before the wait (the paged decode
// step's queries, tables and pools) is written by such kernels only.
#pragma once

#include <cuda_runtime.h>

namespace vfa {

// First statement of a kernel launched this way: nothing after it runs before
// the kernels ahead in the stream have completed.
__device__ __forceinline__ void grid_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// The next kernel of the stream may be scheduled from here on.  Only for a
// kernel whose successor is known to begin with grid_wait(), or to read nothing
// that this one writes (the backward's Delta and dQ kernels): the last kernel
// of a call must not say this, since a decode step behind it reads its pools,
// tables and queries before it waits.
__device__ __forceinline__ void grid_release()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_dependent(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem,
                             cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace vfa
