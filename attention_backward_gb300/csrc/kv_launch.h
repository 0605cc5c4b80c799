// Launch helpers of the paged 8-bit cache operators.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace ab {

// The driver's cuTensorMapEncodeTiled, looked up once (null without a driver).
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Allows ``kern`` ``smem`` bytes of dynamic shared memory on the current device,
// the first time it is asked there (the call costs a microsecond of a launch).
// ``done``: a static of the caller for this kernel, one bit a device.
template <typename... KArgs>
cudaError_t allow_smem_once(void (*kern)(KArgs...), int smem, std::atomic<uint64_t>* done) {
  int dev = 0;
  if (const cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit && (done->load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// launch_after_previous for grids of any shape: ``kern`` may be scheduled
// while the previous kernel on ``st`` finishes, and waits for it with
// grid_dependency_wait before reading its results.
template <typename... KArgs, typename... Args>
cudaError_t launch_chained(void (*kern)(KArgs...), dim3 grid, int threads, int smem, cudaStream_t st,
                           Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace ab
