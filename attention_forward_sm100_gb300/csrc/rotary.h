// Declarations shared by the rotary kernel and its host API.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn_rotary.h"
#include "internal.h"
#include "rotary.cuh"

namespace af {

struct RotaryParams {
  TurnShape shape;             // set by the launch, as block_tokens
  const uint8_t* in[2];        // q, k
  uint8_t* out[2];
  int64_t in_b[2], in_t[2], in_h[2], out_b[2], out_t[2], out_h[2];   // bytes
  const int32_t* positions;
  const int32_t* seqlens;
  const int32_t* cu;           // NULL when fixed
  uint32_t* ws;
  int64_t tokens;              // rows
  int32_t heads[2];
  int32_t batch, seqlen, num_positions;
  int32_t block_tokens;
};

cudaError_t rotary_launch(const RotaryParams& p, int dim, int rot, bool interleaved, bool inverse, const float* table,
                          cudaStream_t stream);

}  // namespace af
