// Rotation of 16-byte pieces (eight bf16) of a head by its token's position.
//
// A pair (x1, x2) becomes (x1 c - x2 s, x2 c + x1 s): two products, each
// rounded, and their sum, rounded; never contracted to a fused multiply-add, so
// that every kernel that rotates gives the same bits.
#pragma once
#include <stdint.h>

#include "ptx.cuh"

namespace af {

// cosines (or sines) of a position, from pair i0 on
template <int N>
__device__ __forceinline__ void load_angles(const float* row, int i0, float (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
    a[i] = v.x;
    a[i + 1] = v.y;
    a[i + 2] = v.z;
    a[i + 3] = v.w;
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) { return __uint_as_float(two & 0xffff0000u); }

// own * c + other * s: the second of a pair; with -s the first (negating a
// product is exact).
__device__ __forceinline__ float turned(float own, float other, float c, float s) {
  return __fadd_rn(__fmul_rn(own, c), __fmul_rn(other, s));
}

// Rotates the E = 8 or 16 values (pieces of eight) that each of the L lanes of a
// vector holds; `x` their bf16 bits, `row` the position's line of the table, of
// `rot` values (a multiple of 16). All lanes of the warp call it; where `on` is
// false the values are only widened.
template <int E, int L>
__device__ __forceinline__ void rotate_lanes(const uint32_t (&x)[E / 2], float (&f)[E], const float* row, int rot,
                                             bool interleaved, bool on) {
  constexpr int P = E / 8;
  const int lane = threadIdx.x % L;
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    f[2 * i] = bf16_lo(x[i]);
    f[2 * i + 1] = bf16_hi(x[i]);
  }
  if (interleaved) {
#pragma unroll
    for (int s = 0; s < P; ++s) {
      const int p = lane * P + s;
      if (on && 8 * p < rot) {
        float c[4], n[4];
        load_angles<4>(row, 4 * p, c);
        load_angles<4>(row, rot / 2 + 4 * p, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = f[8 * s + 2 * i], b = f[8 * s + 2 * i + 1];
          f[8 * s + 2 * i] = turned(a, b, c[i], -n[i]);
          f[8 * s + 2 * i + 1] = turned(b, a, c[i], n[i]);
        }
      }
    }
  } else {
    // the other of piece p's pairs is piece p + half or p - half, in another lane or in this one
    const int half = rot / 16;
#pragma unroll
    for (int s = 0; s < P; ++s) {
      const int p = lane * P + s;
      const bool first = p < half;
      const int q = first ? p + half : (p < 2 * half ? p - half : p);
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t mine = x[4 * s + i];
        if (P == 2 && (half & 1)) mine = x[(4 * (s ^ 1) + i) % (E / 2)];   // (the other slot: half is odd)
        y[i] = __shfl_sync(0xffffffffu, mine, q / P, L);
      }
      if (on && p < 2 * half) {
        float c[8], n[8];
        load_angles<8>(row, 8 * (first ? p : p - half), c);
        load_angles<8>(row, rot / 2 + 8 * (first ? p : p - half), n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = (i & 1) ? bf16_hi(y[i / 2]) : bf16_lo(y[i / 2]);
          f[8 * s + i] = turned(f[8 * s + i], o, c[i], first ? -n[i] : n[i]);
        }
      }
    }
  }
}

}  // namespace af
