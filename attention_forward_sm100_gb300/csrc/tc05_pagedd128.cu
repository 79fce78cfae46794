// Instantiation of the tcgen05 attention kernel for a bf16 paged cache, D = 128.
#include "fa_tc05.cuh"

namespace af {
cudaError_t tc05_launch_pagedd128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream) {
  return tc05_launch_t<TraitsPagedD128>(mask, prm, grid, stream);
}
}  // namespace af
