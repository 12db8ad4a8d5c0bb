// kda_launch.h -- kernel launch with optional programmatic dependent launch.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <utility>

namespace kda {

// Launch `kernel` on `stream`; with `pdl` the kernel may begin while the
// previous kernel in the stream is finishing (it must call pdl_wait() before
// touching that kernel's results).
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem,
                   cudaStream_t stream, bool pdl, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Let `kernel` use `smem` bytes of dynamic shared memory on the current device.  The
// attribute lasts, so each (kernel, device) sets it once (`done`: the kernel's own
// record, by device ordinal).
struct SmemSet {
  std::atomic<unsigned long long> devices{0};
};
template <typename... Params>
cudaError_t allow_smem(void (*kernel)(Params...), size_t smem, SmemSet& done) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = device < 64 ? 1ull << device : 0;
  if (done.devices.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done.devices.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace kda
