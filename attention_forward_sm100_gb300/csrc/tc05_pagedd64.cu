// Instantiation of the tcgen05 attention kernel for a bf16 paged cache, D = 64.
#include "fa_tc05.cuh"

namespace af {
cudaError_t tc05_launch_pagedd64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream) {
  return tc05_launch_t<TraitsPagedD64>(mask, prm, grid, stream);
}
}  // namespace af
