// lq_smem.cu -- the kernels' limit of dynamic shared memory, raised when a launch needs more.
#include <mutex>

#include "lq_internal.cuh"

namespace lq {

// One lock for all kernels: between a look at the cache and its update no other thread may set a
// lower limit, or later calls would trust a limit that is not there. Uncontended it takes some 20 ns.
cudaError_t ensure_smem(const void* func, size_t bytes, int* cache_per_device) {
  if (bytes == 0) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) dev = 0;
  static std::mutex lock;
  const std::lock_guard<std::mutex> held(lock);
  if (cache_per_device[dev] >= (int)bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) cache_per_device[dev] = (int)bytes;
  return e;
}

}  // namespace lq
