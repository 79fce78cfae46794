// What the extension module calls besides the public C ABI.
#pragma once
#include <cuda_runtime_api.h>
#include <stddef.h>

#include "../../include/attn_paged.h"

namespace af {

// attn_paged_fwd with what it needs behind the workspace's first
// ATTN_PAGED_ZEROED_BYTES in memory of its own: at least
// attn_paged_workspace_bytes(p) - ATTN_PAGED_ZEROED_BYTES bytes, 256-byte aligned
// (NULL: behind them, as there).
attn_status paged_fwd(const attn_paged_params* p, void* scratch, size_t scratch_bytes, cudaStream_t stream);

}  // namespace af
