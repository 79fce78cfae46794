// Rows of packed sequences, and the record of what is wrong with them.
#pragma once
#include <stdint.h>

#include "internal.h"

namespace af {

// Records the first invalid length, offset, page or position of a call, of sequence b.
__device__ __forceinline__ void record_error(uint32_t* ws, DeviceError code, int b) {
  if (atomicCAS(&ws[kWsErrorCode], 0u, (uint32_t)code) == 0u) atomicExch(&ws[kWsErrorInfo], (uint32_t)b);
}

// The sequence of row t, for the lanes of the first warp with consecutive rows
// from t0 on (offsets cu[0 .. batch] into `rows` rows); `batch` if it lies behind
// the last one. Every block looks at all offsets: where they decrease, rows cannot
// be told apart, and none has a sequence. The first block records the first
// sequence whose offsets are wrong, whether or not it has a row that is there.
// The whole block of THREADS threads calls it; past kAloneBatch offsets all of its
// warps search (one token each of 1024 sequences, append: 8.8 us with one warp, 6.9
// with all).
constexpr int kAloneBatch = 256;
template <int THREADS>
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t t0, int64_t t, int64_t rows,
                                             uint32_t* ws, DeviceError code) {
  constexpr int WARPS = THREADS / 32;
  __shared__ int part_b[WARPS], part_wrong[WARPS], part_back[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = batch <= kAloneBatch;
  if (alone && warp > 0) return batch;
  int b = 0, wrong = batch;
  bool back = false;
  for (int c = threadIdx.x; c < batch; c += alone ? 32 : THREADS) {
    const int a = cu[c], e = cu[c + 1];
    b += (int64_t)e <= t0 ? 1 : 0;
    back = back || e < a;
    if (a < 0 || e < a || e > rows) wrong = min(wrong, c);
  }
  b = __reduce_add_sync(0xffffffffu, b);
  wrong = __reduce_min_sync(0xffffffffu, wrong);
  back = __any_sync(0xffffffffu, back);
  if (!alone) {
    if (lane == 0) {
      part_b[warp] = b;
      part_wrong[warp] = wrong;
      part_back[warp] = back;
    }
    __syncthreads();
    if (warp > 0) return batch;
    b = __reduce_add_sync(0xffffffffu, lane < WARPS ? part_b[lane] : 0);
    wrong = __reduce_min_sync(0xffffffffu, lane < WARPS ? part_wrong[lane] : batch);
    back = __any_sync(0xffffffffu, lane < WARPS && part_back[lane] != 0);
  }
  if (wrong < batch && blockIdx.x == 0 && lane == 0) record_error(ws, code, wrong);
  if (back) return batch;
  while (b < batch && (int64_t)cu[b + 1] <= t) ++b;
  return b;
}

}  // namespace af
