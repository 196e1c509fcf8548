// Launch attributes that a kernel needs once.
#pragma once

#include <cuda_runtime.h>

#include <atomic>

namespace bsa {

// Dynamic shared memory above 48 KB and clusters above 8 CTAs, asked for once per device (`done`:
// one bit each).
template <typename Kern>
bool allow_smem(Kern kern, int bytes, std::atomic<unsigned long long>& done,
                bool large_cluster = false) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
          cudaSuccess ||
      (large_cluster && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed,
                                             1) != cudaSuccess)) {
    (void)cudaGetLastError();
    return false;
  }
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

}  // namespace bsa
