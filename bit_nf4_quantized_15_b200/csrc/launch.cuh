// Launches of the MXFP4 kernels: shared memory, clusters and programmatic
// dependent launch.
#pragma once

#include <atomic>

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

// The shared-memory attribute (all that a block may have) and that for clusters
// of more than 8 are set once per kernel and device; a launch that fails for
// want of them (the device was reset in between) sets them again.
template <auto* Kern>
cudaError_t allow_big(bool again) {
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!again && (ready.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 232448);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) ready.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <auto* Kern, class... A>
cudaError_t launch_kernel(const LaunchShape& s, cudaStream_t st, const A&... args) {
  const bool big = s.smem > 48 * 1024;
  if (big) {
    const cudaError_t e = allow_big<Kern>(false);
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
  cudaError_t e = cudaLaunchKernelEx(&cfg, Kern, args...);
  if (e == cudaErrorInvalidValue && big && allow_big<Kern>(true) == cudaSuccess) {
    (void)cudaGetLastError();
    e = cudaLaunchKernelEx(&cfg, Kern, args...);
  }
  if (e != cudaSuccess) return e;
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace qnf4
