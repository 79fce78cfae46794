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
#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace af {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;   // vectors a thread has in flight

constexpr int kMaxTokens = 32;   // tokens of a block: one lane each

// Where a token's vectors are in the cache, or page < 0: nowhere.
struct Slot {
  int page, slot;
};

// The sequence of row t, for the lanes of the first warp with consecutive rows
// from t0 on (offsets cu[0 .. batch] into `rows` rows); `batch` if it lies behind
// the last one. Every block looks at all offsets: where they decrease, rows cannot
// be told apart, and none has a sequence. The first block records the first
// sequence whose offsets are wrong, whether or not it has a row that is there.
// The whole block calls it; past kAloneBatch offsets all of its warps search (one
// token each of 1024 sequences, append: 8.8 us with one warp, 6.9 with all).
constexpr int kAloneBatch = 256;
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t t0, int64_t t, int64_t rows,
                                             uint32_t* ws) {
  constexpr int WARPS = kThreads / 32;
  __shared__ int part_b[WARPS], part_wrong[WARPS], part_back[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool alone = batch <= kAloneBatch;
  if (alone && warp > 0) return batch;
  int b = 0, wrong = batch;
  bool back = false;
  for (int c = threadIdx.x; c < batch; c += alone ? 32 : kThreads) {
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
  if (wrong < batch && blockIdx.x == 0 && lane == 0) record_bad_cache(ws, wrong);
  if (back) return batch;
  while (b < batch && (int64_t)cu[b + 1] <= t) ++b;
  return b;
}

__device__ __forceinline__ Slot slot_of(const CacheView& c, int b, int pos, uint32_t* ws) {
  Slot s = {-1, pos & ((1 << c.page_shift) - 1)};
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

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_append_kernel(const __grid_constant__ AppendParams P) {
  constexpr int E = FP8 ? 16 : 8, L = D / E, PER = kThreads / L;
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.tokens - t0);
  const uint32_t nv = 2 * P.c.heads_kv, total = tokens * nv;
  const int lane = threadIdx.x % L;
  // fixed layout: sequence and index of the first token
  const bool packed = P.s.cu_q != nullptr;
  const int b0 = packed ? 0 : (int)((uint32_t)t0 / (uint32_t)P.s.seqlen_q);
  const int i0 = packed ? 0 : (int)t0 - b0 * P.s.seqlen_q;
  auto token_at = [&](int token, int& b, int& i) {
    b = b0;
    i = i0 + token;
    while (i >= P.s.seqlen_q) {
      i -= P.s.seqlen_q;
      ++b;
    }
  };
  for (uint32_t base = 0; base < total; base += PER * kBatch) {
    uint4 x[kBatch][E / 8];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
#pragma unroll
      for (int e = 0; e < E / 8; ++e) x[u][e] = make_uint4(0u, 0u, 0u, 0u);
      if (id < total) {
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        int64_t at;
        if (packed) {
          at = (t0 + w.token) * (w.v ? P.v_t : P.k_t);
        } else {
          int b, i;
          token_at(w.token, b, i);
          at = b * (w.v ? P.v_b : P.k_b) + i * (w.v ? P.v_t : P.k_t);
        }
        const uint8_t* src = (w.v ? P.v + w.h * P.v_h : P.k + w.h * P.k_h) + at + lane * (E * 2);
        if (FP8 && P.wide) {
          ptx::ld_global_v8(src, reinterpret_cast<uint32_t*>(&x[u][0]));
        } else {
#pragma unroll
          for (int e = 0; e < E / 8; ++e) x[u][e] = __ldcs(reinterpret_cast<const uint4*>(src) + e);
        }
      }
    }
    if (base == 0) {
      const int64_t t = t0 + (threadIdx.x & 31);
      const int found = packed ? find_sequence(P.s.cu_q, P.s.batch, t0, t, P.tokens, P.ws) : 0;
      if (threadIdx.x < 32) {
        Slot s = {-1, 0};
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
          token_at(threadIdx.x, b, i);
        }
        if (ok) {
          const int lk = P.s.seqlens_k[b];
          s = slot_of(P.c, b, lk < 0 || lk > P.s.max_k ? -1 : lk - lq + i, P.ws);
        }
        slots[threadIdx.x] = s;
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
      const bool there = id < total;
      const Vector w = vector_at(there ? id : 0u, nv, P.magic, P.c.heads_kv);
      const Slot s = slots[w.token];
      const bool ok = there && s.page >= 0;
      uint8_t* dst = (w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                          : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head) + lane * 16;
      if constexpr (!FP8) {
        if (ok) *reinterpret_cast<uint4*>(dst) = x[u][0];
      } else {
        const uint32_t in[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
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
        const int se = scale_exponent(m);
        const float inv = __uint_as_float((uint32_t)(127 - se) << 23);
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a = in[2 * j], c = in[2 * j + 1];
          out[j] = ptx::pack_e4m3x4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                                    __uint_as_float(c << 16) * inv, __uint_as_float(c & 0xffff0000u) * inv);
        }
        if (ok) {
          *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
          if (lane == 0)
            (w.v ? P.c.v_scale : P.c.k_scale)[(((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot] =
                __uint_as_float((uint32_t)(127 + se) << 23);
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

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr int E = FP8 ? 16 : 8, L = D / E, PER = kThreads / L;
  __shared__ Slot slots[kMaxTokens];
  ptx::grid_dependency_wait();
  const int64_t t0 = (int64_t)blockIdx.x * P.block_tokens;
  const int tokens = (int)min((int64_t)P.block_tokens, P.total_k - t0);
  const uint32_t nv = 2 * P.c.heads_kv, total = tokens * nv;
  const int lane = threadIdx.x % L;
  const int64_t row = t0 + (threadIdx.x & 31);
  const int b = find_sequence(P.cu_k, P.batch, t0, row, P.total_k, P.ws);
  if (threadIdx.x < 32) {
    Slot s = {-1, 0};
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
    uint4 x[kBatch];
    float scale[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
      if (id >= total) continue;
      const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
      const Slot s = slots[w.token];
      if (s.page < 0) continue;
      const uint8_t* src = (w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                                : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head) + lane * 16;
      x[u] = __ldcs(reinterpret_cast<const uint4*>(src));
      if constexpr (FP8)
        scale[u] = __ldg((w.v ? P.c.v_scale : P.c.k_scale) +
                         ((((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot));
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const uint32_t id = base + u * PER + threadIdx.x / L;
      if (id >= total) continue;
      const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
      if (slots[w.token].page < 0) continue;
      const int64_t t = t0 + w.token;
      uint8_t* dst = (w.v ? P.v + t * P.v_t + w.h * P.v_h : P.k + t * P.k_t + w.h * P.k_h) + lane * (E * 2);
      if constexpr (!FP8) {
        *reinterpret_cast<uint4*>(dst) = x[u];
      } else {
        uint32_t out[8];
        widen(x[u], scale[u], out);
        if (P.wide) {
          ptx::st_global_v8(dst, out);
        } else {
          uint4* d = reinterpret_cast<uint4*>(dst);
          d[0] = make_uint4(out[0], out[1], out[2], out[3]);
          d[1] = make_uint4(out[4], out[5], out[6], out[7]);
        }
      }
    }
  }
}

// Every sequence's cached tokens as bf16 pages (WidenParams): blocks (x, b) take
// the token chunks x, x + grid, ... of sequence b. Three bytes of traffic per
// element, HBM bounds it as it does reading.
template <int D>
__global__ void __launch_bounds__(kThreads) cache_widen_kernel(const __grid_constant__ WidenParams P) {
  constexpr int L = D / 16, PER = kThreads / L;
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
      uint4 x[kBatch];
      float scale[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t id = base + u * PER + threadIdx.x / L;
        if (id >= total) continue;
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        const Slot s = slots[w.token];
        if (s.page < 0) continue;
        const uint8_t* src = (w.v ? P.c.v + s.page * P.c.v_page + s.slot * P.c.v_tok + w.h * P.c.v_head
                                  : P.c.k + s.page * P.c.k_page + s.slot * P.c.k_tok + w.h * P.c.k_head) + lane * 16;
        x[u] = __ldg(reinterpret_cast<const uint4*>(src));
        scale[u] = __ldg((w.v ? P.c.v_scale : P.c.k_scale) +
                         ((((int64_t)s.page * P.c.heads_kv + w.h) << P.c.page_shift) + s.slot));
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const uint32_t id = base + u * PER + threadIdx.x / L;
        if (id >= total) continue;
        const Vector w = vector_at(id, nv, P.magic, P.c.heads_kv);
        if (slots[w.token].page < 0) continue;
        const int t = (int)t0 + w.token;
        const int64_t row = (((int64_t)b * P.pages + t / kBlockN) * P.c.heads_kv + w.h) * kBlockN + t % kBlockN;
        uint32_t out[8];
        widen(x[u], scale[u], out);
        ptx::st_global_v8((w.v ? P.v : P.k) + row * (D * 2) + lane * 32, out);
      }
    }
  }
}

// A block's tokens: as many as fill its batch of vectors once.
template <class K, class P>
cudaError_t launch(K kern, P p, int64_t tokens, int vectors, cudaStream_t stream) {
  const uint32_t per_token = 2 * p.c.heads_kv;
  const int fit = vectors / (int)per_token;
  p.block_tokens = fit < 1 ? 1 : (fit < kMaxTokens ? fit : kMaxTokens);
  p.magic = (uint32_t)((((uint64_t)1 << 32) + per_token - 1) / per_token);
  const int64_t blocks = (tokens + p.block_tokens - 1) / p.block_tokens;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_dependent(kern, p, dim3((unsigned)blocks), kThreads, 0, stream);
}

constexpr int per_block(int d, bool fp8) { return kThreads / (d / (fp8 ? 16 : 8)) * kBatch; }

}  // namespace

cudaError_t cache_append_launch(const AppendParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  const int64_t n = p.tokens;
  const int pb = per_block(head_dim, fp8);
  if (head_dim == 128)
    return fp8 ? launch(cache_append_kernel<128, true>, p, n, pb, stream)
               : launch(cache_append_kernel<128, false>, p, n, pb, stream);
  return fp8 ? launch(cache_append_kernel<64, true>, p, n, pb, stream)
             : launch(cache_append_kernel<64, false>, p, n, pb, stream);
}

cudaError_t cache_widen_launch(const WidenParams& params, int head_dim, cudaStream_t stream) {
  WidenParams p = params;
  const uint32_t per_token = 2 * p.c.heads_kv;
  const int fit = per_block(head_dim, true) / (int)per_token;
  p.block_tokens = fit < 1 ? 1 : (fit < kMaxTokens ? fit : kMaxTokens);
  p.magic = (uint32_t)((((uint64_t)1 << 32) + per_token - 1) / per_token);
  const int64_t chunks = ((int64_t)p.max_k + p.block_tokens - 1) / p.block_tokens;
  const int64_t fill = (16ll * sm_count() + p.batch - 1) / p.batch;   // two rounds of eight blocks per SM
  const dim3 grid((unsigned)(chunks < 1 ? 1 : (chunks < fill ? chunks : fill)), (unsigned)p.batch);
  return head_dim == 128 ? launch_dependent(cache_widen_kernel<128>, p, grid, kThreads, 0, stream)
                         : launch_dependent(cache_widen_kernel<64>, p, grid, kThreads, 0, stream);
}

cudaError_t cache_read_launch(const ReadParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  const int64_t n = p.total_k;
  const int pb = per_block(head_dim, fp8);
  if (head_dim == 128)
    return fp8 ? launch(cache_read_kernel<128, true>, p, n, pb, stream)
               : launch(cache_read_kernel<128, false>, p, n, pb, stream);
  return fp8 ? launch(cache_read_kernel<64, true>, p, n, pb, stream)
             : launch(cache_read_kernel<64, false>, p, n, pb, stream);
}

}  // namespace af
