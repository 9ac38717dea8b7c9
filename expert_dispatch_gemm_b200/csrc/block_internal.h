// Host-side helpers of the libmoe_block translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "moe_block.h"

namespace moe {

constexpr int kBlockSms = 148;  // one B200; work splits (and so workspaces) are sized by it

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline moe_status check_block_ws(const void* ws, size_t have, size_t need) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || have < need) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

}  // namespace moe
