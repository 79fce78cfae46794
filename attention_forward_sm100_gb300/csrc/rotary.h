// Declarations shared by the rotary kernel and its host API.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn_rotary.h"
#include "internal.h"

namespace af {

struct RotaryParams {
  const uint8_t* in[2];        // q, k
  uint8_t* out[2];
  int64_t in_b[2], in_t[2], in_h[2], out_b[2], out_t[2], out_h[2];   // bytes
  const float* table;
  const int32_t* positions;
  const int32_t* seqlens;
  const int32_t* cu;           // NULL when fixed
  uint32_t* ws;
  int64_t tokens;              // rows
  int32_t heads[2];
  int32_t batch, seqlen, dim, rot, num_positions;
  int32_t interleaved, inverse;
  int32_t items, slots, block_tokens;   // set by the launch
};

cudaError_t rotary_launch(const RotaryParams& p, cudaStream_t stream);

}  // namespace af
