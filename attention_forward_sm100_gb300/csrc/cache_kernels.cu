// Writing new K/V rows into the paged cache and reading sequences back.
//
// A block takes a few whole tokens (their K and V vectors of all heads). Its first
// warp finds where the tokens live, one lane per token: sequence, position, page.
// The other warps meanwhile load the rows to write; only the stores (when
// reading: the loads) wait for it. A (token, K or V, head) vector is moved by
// D / E lanes, E elements each: 8 for a bf16 cache (16 bytes either way), 16 for
// an e4m3 cache (32 bytes of bf16, 16 bytes of codes). Every byte is moved once
// and next to nothing is computed, so HBM bounds both operations, once the way
// to a vector is short: with the token of each vector found by a 64-bit division
// and its slot looked up by every lane, 190 instructions per vector took 72 us
// for 41690 tokens of 8 heads of 128 (341 MB) where this takes 53.
//
// The 32 bytes of a lane next to an e4m3 cache are one 256-bit access where
// bases and strides allow it (`wide`): as two 16-byte ones, each of a warp's
// accesses touches half of every sector (read of 41690 tokens, 259 MB: 55 us
// against 45).
//
// e4m3: scale = the smallest power of two s with amax / s <= 448. The largest
// finite magnitude is found on the bf16 bit patterns (they order like the
// values) with shuffles inside the vector's lanes; multiplying by 1 / s is
// exact, so the only rounding is the one to e4m3.
//
// e2m1: a lane's sixteen values are one block of the format. s is the smallest
// power of two with amax / s <= 6 * 448, the block's scale e4m3(amax_block / 6 s),
// and a code the rounded quotient x / (s * scale).
//
// With a rotation the keys are turned on their way, in fp32, and the queries of the
// same tokens. Into a bf16 cache all of it is whole rows (append_rows, rotary.cuh);
// where keys are quantised (ROT), a vector's lanes have to meet, and the queries are
// other blocks' work.
#include <type_traits>

#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "rotary.cuh"
#include "rows.cuh"

namespace af {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // vectors a thread has in flight

constexpr int kMaxTokens = 32;   // tokens of a block: one lane each

// Where a token's vectors are in the cache, or page < 0: nowhere. `angle`: its line
// of the rotary table.
struct Slot {
  int page, slot, angle;
};

__device__ __forceinline__ Slot slot_of(const CacheView& c, int b, int pos, uint32_t* ws) {
  Slot s = {-1, pos & ((1 << c.page_shift) - 1), pos};
  if (pos >= 0 && (pos >> c.page_shift) < c.max_pages) {
    const int page = __ldg(c.table + (int64_t)b * c.table_stride + (pos >> c.page_shift));
    if ((unsigned)page < (unsigned)c.num_pages) s.page = page;
  }
  if (s.page < 0) record_bad_cache(ws, b);
  return s;
}

// Vector `idx` of a block: its token and (V behind K) head.
struct Vector {
  int token, h;
  bool v;
};
__device__ __forceinline__ Vector vector_at(uint32_t idx, uint32_t per_token, uint32_t magic, int heads) {
  Vector x;
  x.token = (int)__umulhi(idx, magic);   // idx / per_token (magic = 2^32 / per_token rounded up, idx < 2^16)
  x.h = (int)(idx - x.token * per_token);
  x.v = x.h >= heads;
  if (x.v) x.h -= heads;
  return x;
}

// Largest finite magnitude of two bf16, as 15-bit patterns.
__device__ __forceinline__ uint32_t finite_max(uint32_t two, uint32_t m) {
  const uint32_t lo = two & 0x7fffu, hi = (two >> 16) & 0x7fffu;
  if (lo < 0x7f80u) m = max(m, lo);
  if (hi < 0x7f80u) m = max(m, hi);
  return m;
}

// Exponent of the scale for a largest magnitude of bit pattern `m`.
__device__ __forceinline__ int scale_exponent(uint32_t m) {
  if (m == 0u) return 0;
  const int e = (int)(m >> 7) - 127;             // a subnormal amax ends at the clamp
  return max(-126, e - 8 + ((m & 0x7fu) > 96u ? 1 : 0));   // 1.75 * 2^8 = 448
}

// Exponent of the e2m1 scale for a largest magnitude: of the smallest power of two s
// with m / s <= 6 * 448 = 1.3125 * 2^11.
__device__ __forceinline__ int scale_exponent4(float m) {
  if (m == 0.f) return 0;
  const uint32_t bits = __float_as_uint(m);
  return max(-126, (int)(bits >> 23) - 127 - 11 + ((bits & 0x7fffffu) > 0x280000u ? 1 : 0));
}
// Of the e4m3 scale, for fp32 values.
__device__ __forceinline__ int scale_exponent8(float m) {
  if (m == 0.f) return 0;
  const uint32_t bits = __float_as_uint(m);
  return max(-126, (int)(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0));   // 1.75 * 2^8 = 448
}
__device__ __forceinline__ float finite_max(float x, float m) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? fmaxf(a, m) : m;   // (not infinities and NaN)
}

// e4m3 scale of a block whose largest finite magnitude is `top`, in units of 1 / inv, the
// vector's scale: as its code, and its value.
__device__ __forceinline__ uint32_t block_scale(float top, float inv, float& size) {
  const uint32_t code = ptx::pack_e4m3x4(__fdiv_rn(top * inv, 6.f), 0.f, 0.f, 0.f) & 0xffu;
  float unused;
  ptx::e4m3x2_to_float2(code, size, unused);
  return code;
}
// Sixteen values over a block's scale as e2m1 codes, even ones in the low halves. The
// quotients are correctly rounded, by Markstein's theorem: with r = 1 / size rounded and a
// first quotient t = x r, they are t + r (x - t size), the remainder being exact. Here
// with `size` and r times the vector's scale, 2^se, -100 at least, which changes no
// rounding; two values at a time (57 % of the instructions of one at a time).
__device__ __forceinline__ uint2 quantise_block(const uint64_t (&x)[8], float size, int se) {
  const float r = size == 0.f ? 0.f : __frcp_rn(size);
  const float up = __uint_as_float((uint32_t)(127 - se) << 23) * r, down = -__uint_as_float((uint32_t)(127 + se) << 23) * size;
  const uint64_t r2 = ptx::f2_pack(up, up), s2 = ptx::f2_pack(down, down);
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t first = ptx::f2_mul(x[4 * j + i], r2);
      ptx::f2_unpack(ptx::f2_fma(ptx::f2_fma(first, s2, x[4 * j + i]), r2, first), t[2 * i], t[2 * i + 1]);
    }
    out[j] = ptx::pack_e2m1x8(t);
  }
  return size == 0.f ? make_uint2(0u, 0u) : make_uint2(out[0], out[1]);
}
// The same for any values (infinities, NaN, the smallest scales), one at a time.
__device__ __noinline__ uint2 quantise_any(const float* f, float size, float inv, uint32_t& code) {
  const float r = size == 0.f ? 0.f : __frcp_rn(size);
  uint32_t out[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = f[8 * j + i], y = fminf(fmaxf(x * inv, -2688.f), 2688.f);   // (2688 / size is in range)
      if (x != x) code = 0x7fu;   // a NaN takes its block with it
      t[i] = y * r;
      t[i] = fmaf(fmaf(-t[i], size, y), r, t[i]);
    }
    out[j] = ptx::pack_e2m1x8(t);
  }
  return size == 0.f ? make_uint2(0u, 0u) : make_uint2(out[0], out[1]);
}

// Sequence and index of a block's token, of rows of a fixed length: by a division of
// its own, or counted from the block's first one.
struct TokenByDivision {
  uint32_t t0, len;
  __device__ __forceinline__ TokenByDivision(const AppendParams& P, int64_t t0_)
      : t0((uint32_t)t0_), len((uint32_t)P.s.seqlen_q) {}
  __device__ __forceinline__ void at(int token, int& b, int& i) const {
    const uint32_t t = t0 + (uint32_t)token;
    b = (int)(t / len);
    i = (int)(t - (uint32_t)b * len);
  }
};
struct TokenByCount {
  int b0, i0, len;
  __device__ __forceinline__ TokenByCount(const AppendParams& P, int64_t t0) : b0(0), i0(0), len(P.s.seqlen_q) {
    if (P.s.cu_q != nullptr) return;
    b0 = (int)((uint32_t)t0 / (uint32_t)len);
    i0 = (int)t0 - b0 * len;
  }
  __device__ __forceinline__ void at(int token, int& b, int& i) const {
    b = b0;
    i = i0 + token;
    while (i >= len) {
      i -= len;
      ++b;
    }
  }
};

// Where each of a block's tokens goes (and, ROT, its angle), one lane of the first warp a
// token; ends with a barrier. The whole block calls it.
template <bool ROT, class Params, class Token>
__device__ __forceinline__ void find_slots(const Params& P, int64_t t0, int tokens, const Token& token_of, Slot* slots) {
  const int64_t t = t0 + (threadIdx.x & 31);
  const bool packed = P.s.cu_q != nullptr;
  const int found = packed ? find_sequence<kThreads>(P.s.cu_q, P.s.batch, t0, t, P.tokens, P.ws, kDevErrBadCache) : 0;
  if (threadIdx.x < 32) {
    Slot s = {-1, 0, 0};
    int b, i, lq = P.s.seqlen_q;
    bool ok = (int)threadIdx.x < tokens;
    if (packed) {
      b = found;
      ok = ok && b < P.s.batch;                // else behind the last sequence
      if (ok) {
        const int a = P.s.cu_q[b], e = P.s.cu_q[b + 1];
        i = (int)(t - a);
        lq = e - a;
        // (rows in front of the first sequence; offsets below zero or past
        // the rows, which are recorded)
        ok = a >= 0 && i >= 0 && e <= P.tokens;
      }
    } else {
      token_of.at(threadIdx.x, b, i);
    }
    if (ok) {
      const int lk = P.s.seqlens_k[b];
      s = slot_of(P.c, b, lk < 0 || lk > P.s.max_k ? -1 : lk - lq + i, P.ws);
      if constexpr (ROT) {
        if (P.r.positions != nullptr) s.angle = P.r.positions[t];
        if (s.page >= 0 && (s.angle < 0 || s.angle >= P.r.num_positions)) {
          s.page = -1;
          record_error(P.ws, kDevErrBadPosition, b);
        }
      }
    }
    slots[threadIdx.x] = s;
  }
  __syncthreads();
}

// Offset of a token's rows with batch and token strides sb, st.
template <class Token>
__device__ __forceinline__ int64_t row_offset(const AppendParams& P, int64_t t0, const Token& token_of, int token, int64_t sb,
                                              int64_t st) {
  if (P.s.cu_q != nullptr) return (t0 + token) * st;
  int b, i;
  token_of.at(token, b, i);
  return b * sb + i * st;
}

// The part of an append that moves whole rows, turning keys and queries: the queries of
// any cache, and (KV) keys and values on their way into a bf16 one. Heads are those of
// q, then K's, then V's.
template <bool KV, bool APART>
__device__ __forceinline__ void append_rows(const TurnedAppendParams& P, int block, Slot* slots) {
  const int64_t t0 = (int64_t)block * P.r.block_tokens;
  const int tokens = (int)min((int64_t)P.r.block_tokens, P.tokens - t0);
  const int hq = P.r.heads_q, hkv = P.c.heads_kv;
  const TokenByDivision token_of(P, t0);
  turn_rows<8, APART, kThreads>(
      P.r.shape, tokens,
      [&](int token, int h, TurnHead& head) {
        const uint8_t* base = P.r.q;
        int64_t sb = P.r.q_b, st = P.r.q_t, sh = P.r.q_h;
        if (KV && h >= hq) {
          const bool v = h >= hq + hkv;
          h -= v ? hq + hkv : hq;
          base = v ? P.v : P.k;
          sb = v ? P.v_b : P.k_b;
          st = v ? P.v_t : P.k_t;
          sh = v ? P.v_h : P.k_h;
        }
        head.src = base + row_offset(P, t0, token_of, token, sb, st) + h * sh;
        head.src_next = sh;
      },
      [&]() { find_slots<true>(P, t0, tokens, token_of, slots); },
      [&](int token, int h, TurnHead& head) {
        const Slot s = slots[token];
        if (s.page < 0) return -1;
        if (KV && h >= hq) {
          const bool v = h >= hq + hkv;
          h -= v ? hq + hkv : hq;
          head.dst = v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + h * P.c.v_head
                       : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + h * P.c.k_head;
          head.dst_next = v ? P.c.v_head : P.c.k_head;
        } else {
          head.dst = P.r.q_out + row_offset(P, t0, token_of, token, P.r.out_b, P.r.out_t) + h * P.r.out_h;
          head.dst_next = P.r.out_h;
        }
        return s.angle;
      });
}
// An append with rotation into a bf16 cache: four blocks to an SM (64 registers, a few of
// them spilled). 41690 tokens, 32 query heads and 8 of 128 in the cache, floor 152 us, caches
// flushed, four blocks / three: pairs apart 168 / 186, neighbouring pairs 164 / 160.
template <bool APART>
__global__ void __launch_bounds__(kThreads, 4) append_rows_kernel(const __grid_constant__ TurnedAppendParams P) {
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  append_rows<true, APART>(P, blockIdx.x, slots);
}

template <int D, int KIND, bool ROT>
__global__ void __launch_bounds__(kThreads)
    cache_append_kernel(const __grid_constant__ std::conditional_t<ROT, TurnedAppendParams, AppendParams> P) {
  constexpr int E = KIND == kBf16 ? 8 : 16, L = D / E, PER = kThreads / L;
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  if constexpr (ROT) {
    if ((int)blockIdx.x >= P.blocks_kv) {   // (the queries')
      if (P.r.interleaved) append_rows<false, false>(P, (int)blockIdx.x - P.blocks_kv, slots);
      else append_rows<false, true>(P, (int)blockIdx.x - P.blocks_kv, slots);
      return;
    }
  }
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.tokens - t0);
  const uint32_t nv = 2 * P.c.heads_kv, total = tokens * nv;
  const int lane = threadIdx.x % L;
  const TokenByCount token_of(P, t0);
  for (uint32_t base = 0; base < total; base += PER * kBatch) {
    uint4 x[kBatch][E / 8];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
#pragma unroll
      for (int e = 0; e < E / 8; ++e) x[u][e] = make_uint4(0u, 0u, 0u, 0u);
      if (id < total) {
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        const uint8_t* src = (w.v ? P.v + w.h * P.v_h : P.k + w.h * P.k_h) + lane * (E * 2) +
                             row_offset(P, t0, token_of, w.token, w.v ? P.v_b : P.k_b, w.v ? P.v_t : P.k_t);
        if (KIND != kBf16 && P.wide) {
          ptx::ld_global_v8(src, reinterpret_cast<uint32_t*>(&x[u][0]));
        } else {
#pragma unroll
          for (int e = 0; e < E / 8; ++e) x[u][e] = __ldcs(reinterpret_cast<const uint4*>(src) + e);
        }
      }
    }
    if (base == 0) find_slots<ROT>(P, t0, tokens, token_of, slots);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (base + u * PER >= total) break;
      const uint32_t id = base + u * PER + threadIdx.x / L;
      const bool there = id < total;
      const Vector w = vector_at(there ? id : 0u, nv, P.magic, P.c.heads_kv);
      const Slot s = slots[w.token];
      const bool ok = there && s.page >= 0;
      uint32_t in[E / 2];
#pragma unroll
      for (int e = 0; e < E / 8; ++e) {
        in[4 * e] = x[u][e].x;
        in[4 * e + 1] = x[u][e].y;
        in[4 * e + 2] = x[u][e].z;
        in[4 * e + 3] = x[u][e].w;
      }
      float f[E];
      if constexpr (ROT)
        rotate_lanes<L>(in, f, P.r.table + (int64_t)s.angle * P.r.rot, P.r.rot, P.r.interleaved != 0, ok && !w.v);
      uint8_t* dst = w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                         : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head;
      const int64_t at = (((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot;   // of its scales
      if constexpr (KIND == kBf16) {
        if (ok) *reinterpret_cast<uint4*>(dst + lane * 16) = x[u][0];
      } else if constexpr (KIND == kE4m3) {
        int se;
        if constexpr (ROT) {
          float m = 0.f;
#pragma unroll
          for (int e = 0; e < E; ++e) m = finite_max(f[e], m);
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          se = scale_exponent8(m);
        } else {
          // magnitudes two at a time; only where that meets an infinity or a NaN
          // the finite ones are picked out
          uint32_t m = 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) m = __vmaxu2(m, in[e] & 0x7fff7fffu);
          m = max(m & 0xffffu, m >> 16);
          if (__any_sync(0xffffffffu, m >= 0x7f80u)) {
            m = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = finite_max(in[e], m);
          }
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          se = scale_exponent(m);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[2 * e] = bf16_lo(in[e]);
            f[2 * e + 1] = bf16_hi(in[e]);
          }
        }
        const float inv = __uint_as_float((uint32_t)(127 - se) << 23);
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          out[j] = ptx::pack_e4m3x4(f[4 * j] * inv, f[4 * j + 1] * inv, f[4 * j + 2] * inv, f[4 * j + 3] * inv);
        if (ok) {
          *reinterpret_cast<uint4*>(dst + lane * 16) = make_uint4(out[0], out[1], out[2], out[3]);
          if (lane == 0) (w.v ? P.c.v_scale : P.c.k_scale)[at] = __uint_as_float((uint32_t)(127 + se) << 23);
        }
      } else {
        // the block's largest magnitude, and whether something in it is not finite
        uint64_t pair[8];
        float top = 0.f;
        bool odd;
        if constexpr (ROT) {
          float zero = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            pair[e] = ptx::f2_pack(f[2 * e], f[2 * e + 1]);
            top = ptx::max3(top, fabsf(f[2 * e]), fabsf(f[2 * e + 1]));
            zero = fmaf(f[2 * e], 0.f, fmaf(f[2 * e + 1], 0.f, zero));
          }
          odd = zero != 0.f;
        } else {
          uint32_t m = 0u;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            pair[e] = f2_of(in[e]);
            m = __vmaxu2(m, in[e] & 0x7fff7fffu);
          }
          m = max(m & 0xffffu, m >> 16);
          odd = m >= 0x7f80u;
          top = __uint_as_float(m << 16);
        }
        if (__any_sync(0xffffffffu, odd)) {
          top = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            ptx::f2_unpack(pair[e], f[2 * e], f[2 * e + 1]);
            top = finite_max(f[2 * e], finite_max(f[2 * e + 1], top));
          }
        }
        float m = top;
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        const int se = scale_exponent4(m);
        const float inv = __uint_as_float((uint32_t)(127 - se) << 23);
        float size;
        uint32_t scale = block_scale(top, inv, size);
        uint2 codes;
        if (odd || se < -100) {
          float any[16];
#pragma unroll
          for (int e = 0; e < 8; ++e) ptx::f2_unpack(pair[e], any[2 * e], any[2 * e + 1]);
          codes = quantise_any(any, size, inv, scale);
        } else {
          codes = quantise_block(pair, size, se);
        }
        if (ok) {
          *reinterpret_cast<uint2*>(dst + lane * 8) = codes;
          (w.v ? P.blocks.v : P.blocks.k)[at * L + lane] = (uint8_t)scale;
          if (lane == 0) (w.v ? P.c.v_scale : P.c.k_scale)[at] = __uint_as_float((uint32_t)(127 + se) << 23);
        }
      }
    }
  }
}

// Sixteen codes times their scale, rounded once, as 32 bytes of bf16.
__device__ __forceinline__ void widen(const uint4& x, float scale, uint32_t (&out)[8]) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float2 lo, hi;
    ptx::e4m3x2_to_float2(in[j] & 0xffffu, lo.x, lo.y);
    ptx::e4m3x2_to_float2(in[j] >> 16, hi.x, hi.y);
    out[2 * j] = ptx::pack_bf16(lo.x * scale, lo.y * scale);
    out[2 * j + 1] = ptx::pack_bf16(hi.x * scale, hi.y * scale);
  }
}

// Sixteen values of an e2m1 cache: codes times the block's scale, which is exact,
// times the vector's scale, rounded once.
__device__ __forceinline__ void widen4(const uint2& x, uint32_t block, float scale, uint32_t (&out)[8]) {
  const uint32_t size = ptx::e4m3x2_to_f16x2(block * 0x101u), in[2] = {x.x, x.y};
  const uint64_t s2 = ptx::f2_pack(scale, scale);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t h[4];
    ptx::e2m1x8_to_f16x2(in[j], h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      ptx::f16x2_to_float2(ptx::mul_f16x2(h[i], size), lo, hi);
      ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(lo, hi), s2), lo, hi);
      out[4 * j + i] = ptx::pack_bf16(lo, hi);
    }
  }
}
// Values of a vector that a lane reads: 16 bytes of the cache (e2m1: of 8 bytes a lane,
// finding a vector's place took more instructions than its values: an append of 6360 and
// a read of 38100 tokens, 8 heads of 128, 47.7 us where this takes 45.6).
constexpr int read_width(int kind) { return kind == kBf16 ? 8 : (kind == kE4m3 ? 16 : 32); }
constexpr int read_parts(int kind) { return kind == kE2m1 ? 2 : 1; }   // of sixteen, of a lane's quantised values

// What a lane holds of a quantised vector: its codes and their scales.
template <int KIND>
struct Codes {
  uint4 x;
  uint32_t block;
  float scale;
  // `src`: the vector's first byte, `at` the index of its scales
  __device__ __forceinline__ void load(const uint8_t* src, const float* scales, const uint8_t* blocks, int64_t at,
                                       int lane, int lanes) {
    x = __ldcs(reinterpret_cast<const uint4*>(src + lane * 16));
    if constexpr (KIND == kE2m1) block = __ldg(reinterpret_cast<const uint16_t*>(blocks) + at * lanes + lane);
    scale = __ldg(scales + at);
  }
  __device__ __forceinline__ void widened(int part, uint32_t (&out)[8]) const {
    if constexpr (KIND == kE2m1)
      widen4(part ? make_uint2(x.z, x.w) : make_uint2(x.x, x.y), part ? block >> 8 : block & 0xffu, scale, out);
    else widen(x, scale, out);
  }
};

template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr int E = read_width(KIND), L = D / E, PER = kThreads / L;
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.total_k - t0);
  const uint32_t nv = 2 * P.c.heads_kv, total = tokens * nv;
  const int lane = threadIdx.x % L;
  const int64_t row = t0 + (threadIdx.x & 31);
  const int b = find_sequence<kThreads>(P.cu_k, P.batch, t0, row, P.total_k, P.ws, kDevErrBadCache);
  if (threadIdx.x < 32) {
    Slot s = {-1, 0, 0};
    if ((int)threadIdx.x < tokens && b < P.batch) {
      const int a = P.cu_k[b];
      // (else an offset below zero, which is recorded, or a row in front of the
      // first sequence)
      if (a >= 0 && row >= a) s = slot_of(P.c, b, (int)(row - a), P.ws);
    }
    slots[threadIdx.x] = s;
  }
  __syncthreads();
  for (uint32_t base = 0; base < total; base += PER * kBatch) {
    Codes<KIND> x[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
      if (id >= total) continue;
      const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
      const Slot s = slots[w.token];
      if (s.page < 0) continue;
      const uint8_t* src = w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                               : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head;
      if constexpr (KIND == kBf16)
        x[u].x = __ldcs(reinterpret_cast<const uint4*>(src + lane * 16));
      else
        x[u].load(src, w.v ? P.c.v_scale : P.c.k_scale, w.v ? P.blocks.v : P.blocks.k,
                  (((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot, lane, L);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
      if (id >= total) continue;
      const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
      if (slots[w.token].page < 0) continue;
      const int64_t t = t0 + w.token;
      uint8_t* dst = (w.v ? P.v + t * P.v_t + w.h * P.v_h : P.k + t * P.k_t + w.h * P.k_h) + lane * (E * 2);
      if constexpr (KIND == kBf16) {
        *reinterpret_cast<uint4*>(dst) = x[u].x;
      } else {
#pragma unroll
        for (int part = 0; part < read_parts(KIND); ++part) {
          uint32_t out[8];
          x[u].widened(part, out);
          if (P.wide) {
            ptx::st_global_v8(dst + part * 32, out);
          } else {
            uint4* d = reinterpret_cast<uint4*>(dst) + part * 2;
            d[0] = make_uint4(out[0], out[1], out[2], out[3]);
            d[1] = make_uint4(out[4], out[5], out[6], out[7]);
          }
        }
      }
    }
  }
}

// Every sequence's cached tokens as bf16 pages (WidenParams): blocks (x, b) take
// the token chunks x, x + grid, ... of sequence b. Three bytes of traffic per
// element, HBM bounds it as it does reading.
template <int D, int KIND>
__global__ void __launch_bounds__(kThreads) cache_widen_kernel(const __grid_constant__ WidenParams P) {
  constexpr int L = D / read_width(KIND), PER = kThreads / L;
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  const int b = blockIdx.y, lane = threadIdx.x % L;
  const int lk = min(max(P.seqlens_k[b], 0), P.max_k);   // (a length out of range is recorded by its attention)
  const uint32_t nv = 2 * P.c.heads_kv;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < P.pages; i += kThreads) P.table[(int64_t)b * P.pages + i] = b * P.pages + i;
  const int step = (int)gridDim.x * P.block_tokens;
  for (int64_t t0 = (int64_t)blockIdx.x * P.block_tokens; t0 < lk; t0 += step) {
    const int tokens = (int)min((int64_t)P.block_tokens, lk - t0);
    const uint32_t total = tokens * nv;
    __syncthreads();   // nobody reads the previous chunk's slots any more
    if (threadIdx.x < 32 && (int)threadIdx.x < tokens) slots[threadIdx.x] = slot_of(P.c, b, (int)t0 + threadIdx.x, P.ws);
    __syncthreads();
    for (uint32_t base = 0; base < total; base += PER * kBatch) {
      Codes<KIND> x[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t id = base + u * PER + threadIdx.x / L;
        if (id >= total) continue;
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        const Slot s = slots[w.token];
        if (s.page < 0) continue;
        const uint8_t* src = w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                                 : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head;
        x[u].load(src, w.v ? P.c.v_scale : P.c.k_scale, w.v ? P.blocks.v : P.blocks.k,
                  (((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot, lane, L);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t id = base + u * PER + threadIdx.x / L;
        if (id >= total) continue;
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        if (slots[w.token].page < 0) continue;
        const int t = (int)t0 + w.token;
        const int64_t row = (((int64_t)b * P.pages + t / kBlockN) * P.c.heads_kv + w.h) * kBlockN + t % kBlockN;
#pragma unroll
        for (int part = 0; part < read_parts(KIND); ++part) {
          uint32_t out[8];
          x[u].widened(part, out);
          ptx::st_global_v8((w.v ? P.v : P.k) + row * (D * 2) + (lane * read_parts(KIND) + part) * 32, out);
        }
      }
    }
  }
}

// A block's tokens: as many as fill its batch of vectors once, at most (FEW) as leave
// no SM without a block: values to quantise are one vector's after another's in a thread.
// (32 tokens, 32 query heads and 8 of 128 in the cache, e2m1 with rotation: 13 us with
// eight tokens to a block, 6 with one. What is only moved is not faster in smaller blocks:
// 96 tokens of 8 heads, bf16, 3.6 us with four, 3.7 with one.)
template <bool FEW>
int tokens_of_block(int64_t tokens, uint32_t per_token, int vectors) {
  const int64_t fit = vectors / (int)per_token, few = FEW ? tokens / sm_count() : fit;
  const int64_t n = fit < few ? fit : few;
  return n < 1 ? 1 : (n < kMaxTokens ? (int)n : kMaxTokens);
}
template <bool FEW = false, class K, class P>
cudaError_t launch(K kern, P p, int64_t tokens, uint32_t per_token, int vectors, cudaStream_t stream) {
  p.block_tokens = tokens_of_block<FEW>(tokens, per_token, vectors);
  p.magic = (uint32_t)((((uint64_t)1 << 32) + per_token - 1) / per_token);
  const int64_t blocks = (tokens + p.block_tokens - 1) / p.block_tokens;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_dependent(kern, p, dim3((unsigned)blocks), kThreads, 0, stream);
}

constexpr int per_block(int d, int kind) { return kThreads / (d / (kind == kBf16 ? 8 : 16)) * kBatch; }
constexpr int read_block(int d, int kind) { return kThreads / (d / read_width(kind)) * kBatch; }

// Rows to be turned: blocks of them, with their sizes in `p`.
int64_t turn_blocks(TurnedAppendParams& p, int head_dim, const int (&heads)[3], int turned) {
  AppendRotary& r = p.r;
  r.shape = turn_shape(r.table, head_dim, r.rot, r.interleaved != 0, false, heads, turned);
  r.block_tokens = turn_tokens(r.shape, p.tokens, kThreads, kMaxTokens, sm_count());
  return (p.tokens + r.block_tokens - 1) / r.block_tokens;
}

template <int D, int KIND>
cudaError_t append_t(const TurnedAppendParams& params, cudaStream_t stream) {
  TurnedAppendParams p = params;
  const uint32_t per_token = 2 * p.c.heads_kv;
  const int vectors = per_block(D, KIND);
  if (p.r.table == nullptr)
    return launch<KIND == kE2m1>(cache_append_kernel<D, KIND, false>, static_cast<const AppendParams&>(params), p.tokens,
                                 per_token, vectors, stream);
  if constexpr (KIND == kBf16) {
    const int64_t blocks = turn_blocks(p, D, {p.r.heads_q, p.c.heads_kv, p.c.heads_kv}, 2);
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    return turn_apart(p.r.shape) ? launch_dependent(append_rows_kernel<true>, p, grid, kThreads, 0, stream)
                                 : launch_dependent(append_rows_kernel<false>, p, grid, kThreads, 0, stream);
  } else {
    const int64_t rows = p.r.heads_q > 0 ? turn_blocks(p, D, {p.r.heads_q, 0, 0}, 1) : 0;
    p.block_tokens = tokens_of_block<true>(p.tokens, per_token, vectors);
    p.magic = (uint32_t)((((uint64_t)1 << 32) + per_token - 1) / per_token);
    const int64_t blocks = (p.tokens + p.block_tokens - 1) / p.block_tokens;
    if (blocks + rows > 0x7fffffffll) return cudaErrorInvalidValue;
    p.blocks_kv = (int32_t)blocks;
    return launch_dependent(cache_append_kernel<D, KIND, true>, p, dim3((unsigned)(blocks + rows)), kThreads, 0, stream);
  }
}
template <int D>
cudaError_t append_d(const TurnedAppendParams& p, int kind, cudaStream_t stream) {
  return kind == kBf16 ? append_t<D, kBf16>(p, stream)
                       : (kind == kE4m3 ? append_t<D, kE4m3>(p, stream) : append_t<D, kE2m1>(p, stream));
}
template <int D>
cudaError_t read_d(const ReadParams& p, int kind, cudaStream_t stream) {
  const uint32_t n = 2 * p.c.heads_kv;
  const int pb = read_block(D, kind);
  return kind == kBf16 ? launch(cache_read_kernel<D, kBf16>, p, p.total_k, n, pb, stream)
                       : (kind == kE4m3 ? launch(cache_read_kernel<D, kE4m3>, p, p.total_k, n, pb, stream)
                                        : launch(cache_read_kernel<D, kE2m1>, p, p.total_k, n, pb, stream));
}
template <int D>
cudaError_t widen_d(const WidenParams& p, int kind, dim3 grid, cudaStream_t stream) {
  return kind == kE4m3 ? launch_dependent(cache_widen_kernel<D, kE4m3>, p, grid, kThreads, 0, stream)
                       : launch_dependent(cache_widen_kernel<D, kE2m1>, p, grid, kThreads, 0, stream);
}

}  // namespace

cudaError_t cache_append_launch(const TurnedAppendParams& p, int head_dim, int kind, cudaStream_t stream) {
  return head_dim == 128 ? append_d<128>(p, kind, stream) : append_d<64>(p, kind, stream);
}

cudaError_t cache_widen_launch(const WidenParams& params, int head_dim, int kind, cudaStream_t stream) {
  WidenParams p = params;
  const uint32_t per_token = 2 * p.c.heads_kv;
  const int fit = read_block(head_dim, kind) / (int)per_token;
  p.block_tokens = fit < 1 ? 1 : (fit < kMaxTokens ? fit : kMaxTokens);
  p.magic = (uint32_t)((((uint64_t)1 << 32) + per_token - 1) / per_token);
  const int64_t chunks = ((int64_t)p.max_k + p.block_tokens - 1) / p.block_tokens;
  const int64_t fill = (16ll * sm_count() + p.batch - 1) / p.batch;   // two rounds of eight blocks per SM
  const dim3 grid((unsigned)(chunks < 1 ? 1 : (chunks < fill ? chunks : fill)), (unsigned)p.batch);
  return head_dim == 128 ? widen_d<128>(p, kind, grid, stream) : widen_d<64>(p, kind, grid, stream);
}

cudaError_t cache_read_launch(const ReadParams& p, int head_dim, int kind, cudaStream_t stream) {
  return head_dim == 128 ? read_d<128>(p, kind, stream) : read_d<64>(p, kind, stream);
}

}  // namespace af
