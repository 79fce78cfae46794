// Queries and keys turned by their positions (attn_rotary.h); rotary.cuh has the work
// on the rows.
#include "launch.cuh"
#include "rotary.cuh"
#include "rotary.h"
#include "rows.cuh"

namespace af {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;   // tokens of a block: one lane each

// Position of each of the block's tokens, -1 for one that is not written. The
// whole block calls it.
__device__ __forceinline__ void find_positions(const RotaryParams& P, int64_t t0, int tokens, int* at) {
  const int64_t t = t0 + (threadIdx.x & 31);
  int b = P.batch, i = 0, n = P.seqlen;
  const bool packed = P.cu != nullptr;
  if (packed)
    b = find_sequence<kThreads>(P.cu, P.batch, t0, t, P.tokens, P.ws, kDevErrBadPosition);
  else if (threadIdx.x < 32)
    b = (int)((uint32_t)t / (uint32_t)P.seqlen), i = (int)((uint32_t)t - (uint32_t)b * (uint32_t)P.seqlen);
  if (threadIdx.x < 32) {
    int pos = -1;
    if ((int)threadIdx.x < tokens && b < P.batch) {
      bool there = true;
      if (packed) {
        const int a = P.cu[b], e = P.cu[b + 1];
        i = (int)(t - a);
        n = e - a;
        there = a >= 0 && i >= 0 && e <= P.tokens;   // (else recorded, or a row in front of the first sequence)
      }
      if (there) {
        int64_t p = i;
        if (P.positions != nullptr) p = P.positions[t];
        else if (P.seqlens != nullptr) p = (int64_t)P.seqlens[b] - n + i;
        if (p >= 0 && p < P.num_positions) pos = (int)p;
        else record_error(P.ws, kDevErrBadPosition, b);
      }
    }
    at[threadIdx.x] = pos;
  }
  __syncthreads();
}

// (Pairs apart at four blocks to an SM, 64 registers and a few of them spilled: 41690 tokens,
// 40 heads of 128, 147 us instead of 151, half of each head turned 183 instead of 195.)
template <int W, bool APART>
__global__ void __launch_bounds__(kThreads, W == 8 && APART ? 4 : 3) rotary_kernel(const __grid_constant__ RotaryParams P) {
  __shared__ int positions[kMaxTokens];
  ptx::grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.tokens - t0);
  // the first head of (token, h) among rows with these strides
  auto row = [&](int token, const int64_t (&sb)[2], const int64_t (&st)[2], int which) -> int64_t {
    const uint32_t t = (uint32_t)(t0 + token);
    if (P.cu != nullptr) return t * st[which];
    const uint32_t b = t / (uint32_t)P.seqlen;
    return b * sb[which] + (t - b * (uint32_t)P.seqlen) * st[which];
  };
  turn_rows<W, APART, kThreads>(
      P.shape, tokens,
      [&](int token, int h, TurnHead& head) {
        const int which = h >= P.heads[0] ? 1 : 0;
        head.src = P.in[which] + row(token, P.in_b, P.in_t, which) + (which ? h - P.heads[0] : h) * P.in_h[which];
        head.src_next = P.in_h[which];
      },
      [&]() { find_positions(P, t0, tokens, positions); },
      [&](int token, int h, TurnHead& head) {
        const int which = h >= P.heads[0] ? 1 : 0;
        head.dst = P.out[which] + row(token, P.out_b, P.out_t, which) + (which ? h - P.heads[0] : h) * P.out_h[which];
        head.dst_next = P.out_h[which];
        return positions[token];
      });
}

}  // namespace

cudaError_t rotary_launch(const RotaryParams& params, int dim, int rot, bool interleaved, bool inverse, const float* table,
                          cudaStream_t stream) {
  RotaryParams p = params;
  p.shape = turn_shape(table, dim, rot, interleaved, inverse, {p.heads[0], p.heads[1], 0}, 2);
  p.block_tokens = turn_tokens(p.shape, p.tokens, kThreads, kMaxTokens, sm_count());
  const int64_t blocks = (p.tokens + p.block_tokens - 1) / p.block_tokens;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks);
  if (!turn_apart(p.shape)) return launch_dependent(rotary_kernel<8, false>, p, grid, kThreads, 0, stream);
  return turn_wide(p.shape) ? launch_dependent(rotary_kernel<8, true>, p, grid, kThreads, 0, stream)
                            : launch_dependent(rotary_kernel<1, true>, p, grid, kThreads, 0, stream);
}

}  // namespace af
