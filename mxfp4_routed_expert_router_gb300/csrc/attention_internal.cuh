// attention_internal.cuh -- what the files of the attention operators share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "moe_internal.cuh"

namespace moe {

constexpr int ATTN_MAX_HEADS = 1024;

// The attention operators have no handle: kernels record what goes wrong in one flag per device (the first error
// stays until moe_attention_status takes it).  Its address on the current device, or an error.
cudaError_t attention_error_flag(int **flag);

// MOE_OK, or the status (with its message set) of what is wrong with a cache.
MoeStatus check_kv_cache(const MoeKvCache *c);

inline bool rows_16b(const void *p, long long ld) { return (uintptr_t)p % 16 == 0 && ld * 2 % 16 == 0; }

}  // namespace moe
