// Several kernels of one call in a row (programmatic dependent launch).
#pragma once

#include <cuda_runtime.h>

namespace gecko {

// A call's kernels overlap at their ends: each lets the next one start as soon as
// all its own blocks run, and waits for the one before (and so for all before that)
// before it touches global memory, with barriers and TMEM set up by then.  A call's
// first kernel is launched without the attribute.  The projection's gradients at
// 777 x 520 x 1032 in fp32, five kernels: 47 us a call without this, 40 with it; 512
// x 512 x 512 in bf16 31 and 25.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// `after`: another kernel of the same call is before this one on the stream.
template <class... P, class... A>
cudaError_t launch_chained(void (*kern)(P...), dim3 grid, int threads, int smem, int cluster, bool after,
                           cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (cluster) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

}  // namespace gecko
