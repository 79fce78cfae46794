// Queries and keys turned by their positions (attn_rotary.h).
//
// Every byte of q and k moves once each way, and a token's line of the table
// (4 R bytes, for all its heads) once from L2: HBM bounds it. A thread takes one
// item of a token, an item being what is turned together: 16 bytes and, in the
// half layout, the 16 bytes R / 2 behind them (or 16 bytes that are only
// copied). It keeps the item's cosines and sines in registers and goes through
// kHeads heads, whose loads are all in flight before the first is used.
// Tables or depths that pieces of eight do not fit are done value by value
// (W = 1).
#include "launch.cuh"
#include "rotary.cuh"
#include "rotary.h"
#include "rows.cuh"

namespace af {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 4;        // heads of a thread
constexpr int kMaxTokens = 32;   // tokens of a block: one lane each

// W values that lie together.
template <int W>
struct Values;
template <>
struct Values<8> {
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void store(uint8_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(w[i]);
      f[2 * i + 1] = bf16_hi(w[i]);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    v = make_uint4(ptx::pack_bf16(f[0], f[1]), ptx::pack_bf16(f[2], f[3]), ptx::pack_bf16(f[4], f[5]),
                   ptx::pack_bf16(f[6], f[7]));
  }
};
template <>
struct Values<1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = *reinterpret_cast<const uint16_t*>(p); }
  __device__ __forceinline__ void store(uint8_t* p) const { *reinterpret_cast<uint16_t*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = __uint_as_float((uint32_t)v << 16); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = (uint16_t)ptx::pack_bf16(f[0], 0.f); }
};

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

template <int W>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryParams P) {
  __shared__ int positions[kMaxTokens];
  ptx::grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.tokens - t0);
  find_positions(P, t0, tokens, positions);
  const int per_token = P.items * P.slots;
  // Pieces of eight of the interleaved layout hold both values of their pairs; else
  // the first `half` items have two parts.
  const bool apart = W == 1 || !P.interleaved;
  const int half = apart ? P.rot / 2 / W : 0;
  const int heads = P.heads[0] + P.heads[1];
  for (int x = threadIdx.x; x < tokens * per_token; x += kThreads) {
    const int token = x / per_token, rest = x - token * per_token;
    const int slot = rest / P.items, item = rest - slot * P.items;
    const int pos = positions[token];
    if (pos < 0) continue;
    const uint32_t t = (uint32_t)(t0 + token);
    const int64_t b = P.cu != nullptr ? 0 : t / (uint32_t)P.seqlen;
    const int64_t i = P.cu != nullptr ? t : t - (uint32_t)b * (uint32_t)P.seqlen;
    const bool pair = item < half;
    // first value of the item, and of its other part
    int d = (pair || !apart ? item : item + half) * W, d2 = d + P.rot / 2;
    if (W == 1 && pair && P.interleaved) {
      d = 2 * item;
      d2 = d + 1;
    }
    Values<W> u[kHeads], w[kHeads];
    uint8_t* dst[kHeads];
#pragma unroll
    for (int y = 0; y < kHeads; ++y) {
      int h = slot + y * P.slots;
      dst[y] = nullptr;
      if (h >= heads) continue;
      const int which = h >= P.heads[0] ? 1 : 0;
      if (which) h -= P.heads[0];
      const uint8_t* src = (which ? P.in[1] + b * P.in_b[1] + i * P.in_t[1] + h * P.in_h[1]
                                  : P.in[0] + b * P.in_b[0] + i * P.in_t[0] + h * P.in_h[0]);
      dst[y] = (which ? P.out[1] + b * P.out_b[1] + i * P.out_t[1] + h * P.out_h[1]
                      : P.out[0] + b * P.out_b[0] + i * P.out_t[0] + h * P.out_h[0]);
      u[y].load(src + 2 * d);
      if (pair) w[y].load(src + 2 * d2);
    }
    const float* row = P.table + (int64_t)pos * P.rot;
    if (pair) {
      float c[W], n[W];
      if constexpr (W == 8) {
        load_angles<W>(row, d, c);
        load_angles<W>(row, P.rot / 2 + d, n);
      } else {
        c[0] = __ldg(row + item);
        n[0] = __ldg(row + P.rot / 2 + item);
      }
#pragma unroll
      for (int y = 0; y < kHeads; ++y) {
        if (dst[y] == nullptr) continue;
        float f[W], g[W], f2[W], g2[W];
        u[y].get(f);
        w[y].get(g);
#pragma unroll
        for (int j = 0; j < W; ++j) {
          const float s = P.inverse ? -n[j] : n[j];
          f2[j] = turned(f[j], g[j], c[j], -s);
          g2[j] = turned(g[j], f[j], c[j], s);
        }
        u[y].set(f2);
        w[y].set(g2);
        u[y].store(dst[y] + 2 * d);
        w[y].store(dst[y] + 2 * d2);
      }
    } else {
      if constexpr (W == 8) {
        if (!apart && d < P.rot) {
          float c[4], n[4];
          load_angles<4>(row, d / 2, c);
          load_angles<4>(row, P.rot / 2 + d / 2, n);
#pragma unroll
          for (int y = 0; y < kHeads; ++y) {
            if (dst[y] == nullptr) continue;
            float f[8];
            u[y].get(f);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float s = P.inverse ? -n[j] : n[j], a = f[2 * j], e = f[2 * j + 1];
              f[2 * j] = turned(a, e, c[j], -s);
              f[2 * j + 1] = turned(e, a, c[j], s);
            }
            u[y].set(f);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < kHeads; ++y)
        if (dst[y] != nullptr) u[y].store(dst[y] + 2 * d);
    }
  }
}

}  // namespace

cudaError_t rotary_launch(const RotaryParams& params, cudaStream_t stream) {
  RotaryParams p = params;
  const bool wide = p.rot % (p.interleaved ? 8 : 16) == 0;
  const int w = wide ? 8 : 1;
  p.items = wide && p.interleaved ? p.dim / w : p.dim / w - p.rot / 2 / w;
  const int heads = p.heads[0] + p.heads[1];
  p.slots = (heads + kHeads - 1) / kHeads;
  const int64_t per_token = (int64_t)p.items * p.slots;
  const int64_t fit = kThreads / per_token;
  p.block_tokens = fit < 1 ? 1 : (fit < kMaxTokens ? (int)fit : kMaxTokens);
  const int64_t blocks = (p.tokens + p.block_tokens - 1) / p.block_tokens;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return wide ? launch_dependent(rotary_kernel<8>, p, dim3((unsigned)blocks), kThreads, 0, stream)
              : launch_dependent(rotary_kernel<1>, p, dim3((unsigned)blocks), kThreads, 0, stream);
}

}  // namespace af
