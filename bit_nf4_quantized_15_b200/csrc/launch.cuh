// Launches of the MXFP4 kernels: shared memory, clusters and programmatic
// dependent launch.
#pragma once

#include "common.cuh"
#include "internal.h"

namespace qnf4 {

// Lets the next kernel of the call start its prologue now; it waits
// (pdl_wait) for this one to finish before it touches what this one writes.
QDEV void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
// Until the kernel before this one has finished and its writes are visible
// (at once in a launch without the attribute).
QDEV void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

struct LaunchShape {
  dim3 grid;
  unsigned threads;
  size_t smem;
  unsigned cluster;  // 1: none (or the kernel's own)
  bool dependent;    // starts while the kernel before it on the stream still runs
};

template <class K, class... A>
cudaError_t launch_kernel(K* kern, const LaunchShape& s, cudaStream_t st, const A&... args) {
  if (s.smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)s.smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = s.grid;
  cfg.blockDim = dim3(s.threads);
  cfg.dynamicSmemBytes = s.smem;
  cfg.stream = st;
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (s.cluster > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = s.cluster;
    at[n].val.clusterDim.y = 1;
    at[n++].val.clusterDim.z = 1;
  }
  if (s.dependent) {
    at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[n++].val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = at;
  cfg.numAttrs = n;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
