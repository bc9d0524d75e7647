// Grid of a persistent kernel: the CTAs that the current device runs at once.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace ssd {

// What a kernel's launcher keeps of each device (0: not yet asked for); a
// kernel's threads and shared memory do not change from call to call.
struct FitOf {
  static constexpr int kDevices = 64;
  std::atomic<int> fit[kDevices] = {};
};

// At most `cap` CTAs and no more than there are steps.  The kernel's limit of
// shared memory is set in every call: it belongs to the device's context.
template <typename KernelT>
cudaError_t persistent_grid(KernelT kernel, int threads, size_t smem, long long steps, int cap,
                            FitOf* keep, int* grid) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < FitOf::kDevices;
  int n = kept ? keep->fit[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    int nsm = 0, occ = 0;
    e = cudaDeviceGetAttribute(&nsm, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    n = nsm * (occ > 0 ? occ : 1);
    if (kept) keep->fit[dev].store(n, std::memory_order_relaxed);
  }
  if (n > cap) n = cap;
  *grid = (int)(steps < n ? steps : n);
  return cudaSuccess;
}

}  // namespace ssd
