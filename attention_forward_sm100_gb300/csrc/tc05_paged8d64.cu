// Instantiation of the tcgen05 attention kernel for an e4m3 paged cache, D = 64.
#include "fa_tc05.cuh"

namespace af {
cudaError_t tc05_launch_paged8d64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream) {
  return tc05_launch_t<TraitsPaged8D64>(mask, prm, grid, stream);
}
}  // namespace af
