// smem_limit.h -- kernels' limits of dynamic shared memory (host code; needs the
// declarations of the CUDA runtime only).
#pragma once

#include <cuda_runtime_api.h>
#include <stddef.h>

#include <atomic>

namespace moe {

// Lets `kern` use `bytes` of dynamic shared memory.  done: a flag for each device,
// kept by the caller for each kernel, so that only its first call asks.
// The limit is set to all that a block of the kernel can have, whatever this call
// needs: calls of several host threads then set the same value, and none lowers what
// another has asked for.
struct SmemAllowed {
  std::atomic<bool> device[64];  // (zero: objects of static storage)
};
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, SmemAllowed& done) {
  if (bytes <= 40 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < 64;
  if (known && done.device[dev].load(std::memory_order_acquire)) return cudaSuccess;
  const void* f = reinterpret_cast<const void*>(kern);
  cudaFuncAttributes a;
  int most = 0;
  e = cudaFuncGetAttributes(&a, f);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, most - (int)a.sharedSizeBytes);
  if (e == cudaSuccess && known) done.device[dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace moe
