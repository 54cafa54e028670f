// Host helpers of kernel launches: shared-memory opt-in and launches that may
// begin while the one before ends.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "longnet.h"

namespace longnet {

// Opts a kernel in to its shared memory, once per device (fn's instantiations
// have a flag each).
template <auto fn>
bool opt_in_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return false;
  }
  if ((done.load(std::memory_order_acquire) >> dev) & 1) return true;
  if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.fetch_or((uint64_t)1 << dev, std::memory_order_release);
  return true;
}

template <typename... P, typename... V>
int launch_after(void (*fn)(P...), dim3 grid, int threads, int smem, cudaStream_t stream, V&&... args) {
  // programmatic dependent launch: the kernel's set-up overlaps the end of the
  // launch before it, whose results it waits for (griddepcontrol.wait)
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
  if (cudaLaunchKernelEx(&cfg, fn, args...) != cudaSuccess) {
    cudaGetLastError();
    return LONGNET_ERR_CUDA;
  }
  return LONGNET_OK;
}

}  // namespace longnet
