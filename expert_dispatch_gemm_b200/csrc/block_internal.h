// Host-side helpers of the libmoe_block translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "moe_block.h"

namespace moe {

constexpr int kBlockSms = 148;  // one B200; work splits (and so workspaces) are sized by it

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline moe_status check_block_ws(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || have < need) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Raises the kernel's shared-memory limit to `bytes`, once on each device. The
// limit belongs to the kernel, not to a launch: `bytes` has to be the most that any
// launch of it takes, or a thread would lower what another is about to launch
// with. `done`: a static of the kernel's.
template <class K>
inline cudaError_t allow_smem(K kern, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace moe
