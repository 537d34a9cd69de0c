// launch.h - what a kernel's launches share.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace fa {

// Sets a kernel's dynamic shared memory once on each device (`done`: one bit per
// device id; ids past 63 set it on every launch): the attribute calls of a small
// backward pass took 1.5 us of its 40 us on the host.
template <typename Kernel>
inline cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<unsigned long long> &done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? (1ull << dev) : 0ull;
  if (bit != 0ull && (done.load(std::memory_order_acquire) & bit) != 0ull) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace fa
