// launch.cuh -- launching kernels that overlap the end of the one before.
//
// A kernel launched by launch_chained may start while the stream's previous
// kernel still runs: its blocks set up their barriers and shared memory and
// then wait (chain_wait) until everything before them in the stream is
// complete and visible.  Every block of such a kernel passes chain_wait before
// it touches anything that another kernel reads or writes, on every path: what
// follows in the stream relies on this kernel's end coming after the end of
// what it waited for.  What it reads may still be written while it starts, so
// that is read by ordinary loads, none of the read-only path's.  chain_next lets
// the next kernel's blocks come as soon as this one's leave room.  Back to back,
// short kernels start 2 us earlier so.
#pragma once

#include <cuda_runtime.h>

namespace tsm {

__device__ __forceinline__ void chain_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void chain_next()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// `cluster` 0: no cluster attribute.
template <typename... P, typename... A>
cudaError_t launch_chained(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster,
                           cudaStream_t stream, const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace tsm
