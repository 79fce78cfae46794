// Writing new K/V rows into the paged cache and reading sequences back.
//
// One (token, K or V, head) vector is handled by D / E lanes, each moving E
// elements: 8 for a bf16 cache (16 bytes either way), 16 for an e4m3 cache
// (32 bytes of bf16, 16 bytes of codes). Both operations move every byte once
// and compute next to nothing, so HBM bounds them; what the kernels add is the
// way from a row to its slot (sequence, position, page), done per vector from
// L1/L2-resident tables while the vector itself is on its way.
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

// Sequence that holds row t: the number of sequences that end at or before t
// (offsets cu[0..batch]). All threads of the block, with one barrier.
__device__ __forceinline__ int find_sequence(const int32_t* cu, int batch, int64_t t) {
  int n = 0;
  for (int b = threadIdx.x; b < batch; b += kThreads) n += (int64_t)cu[b + 1] <= t ? 1 : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  __shared__ int part[kThreads / 32];
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) n += part[w];
  return n;
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
  ptx::grid_dependency_wait();
  const int nv = 2 * P.c.heads_kv;               // vectors of one token
  const int64_t total = P.tokens * nv;
  const int64_t first = (int64_t)blockIdx.x * (PER * kBatch);
  const int lane = threadIdx.x % L;
  int b0 = 0;
  if (P.s.cu_q != nullptr) b0 = find_sequence(P.s.cu_q, P.s.batch, first / nv);
  uint4 x[kBatch][E / 8];
  uint8_t* dst[kBatch];
  float* sdst[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    dst[u] = nullptr;
    sdst[u] = nullptr;
    const int64_t id = first + u * PER + threadIdx.x / L;
#pragma unroll
    for (int e = 0; e < E / 8; ++e) x[u][e] = make_uint4(0u, 0u, 0u, 0u);
    if (id >= total) continue;
    const int64_t t = id / nv;
    const int w = (int)(id - t * nv);
    const bool is_v = w >= P.c.heads_kv;
    const int h = is_v ? w - P.c.heads_kv : w;
    int b, i;
    if (P.s.cu_q == nullptr) {
      b = (int)(t / P.s.seqlen_q);
      i = (int)(t - (int64_t)b * P.s.seqlen_q);
    } else {
      b = b0;
      while (b < P.s.batch && (int64_t)P.s.cu_q[b + 1] <= t) ++b;
      if (b >= P.s.batch) continue;              // behind the last sequence
      i = (int)(t - P.s.cu_q[b]);
    }
    const uint8_t* src = (is_v ? P.v + (int64_t)h * P.v_h : P.k + (int64_t)h * P.k_h) +
                         (P.s.cu_q == nullptr ? b * (is_v ? P.v_b : P.k_b) + i * (is_v ? P.v_t : P.k_t)
                                              : t * (is_v ? P.v_t : P.k_t)) + lane * (E * 2);
#pragma unroll
    for (int e = 0; e < E / 8; ++e) x[u][e] = __ldcs(reinterpret_cast<const uint4*>(src) + e);
    // the slot: position, then page
    const int a = P.s.cu_q == nullptr ? 0 : P.s.cu_q[b];
    const int lq = P.s.cu_q == nullptr ? P.s.seqlen_q : P.s.cu_q[b + 1] - a;
    const int lk = P.s.seqlens_k[b];
    const int pos = lk - lq + i;
    if (a < 0 || i < 0 || i >= lq || lk > P.s.max_k || pos < 0) {
      record_bad_cache(P.ws, b);
      continue;
    }
    const int page = __ldg(P.c.table + (int64_t)b * P.c.table_stride + (pos >> P.c.page_shift));
    if ((unsigned)page >= (unsigned)P.c.num_pages) {
      record_bad_cache(P.ws, b);
      continue;
    }
    const int slot = pos & ((1 << P.c.page_shift) - 1);
    dst[u] = (is_v ? P.c.v + page * P.c.v_page + slot * P.c.v_tok + h * P.c.v_head
                   : P.c.k + page * P.c.k_page + slot * P.c.k_tok + h * P.c.k_head) + lane * 16;
    if constexpr (FP8)
      sdst[u] = (is_v ? P.c.v_scale : P.c.k_scale) +
                ((((int64_t)page * P.c.heads_kv + h) << P.c.page_shift) + slot);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    if constexpr (!FP8) {
      if (dst[u] != nullptr) *reinterpret_cast<uint4*>(dst[u]) = x[u][0];
    } else {
      uint32_t m = 0u;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m = finite_max(x[u][e].x, m);
        m = finite_max(x[u][e].y, m);
        m = finite_max(x[u][e].z, m);
        m = finite_max(x[u][e].w, m);
      }
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
      const int se = scale_exponent(m);
      const float inv = __uint_as_float((uint32_t)(127 - se) << 23);
      uint32_t out[4];
      const uint32_t* in = reinterpret_cast<const uint32_t*>(&x[u][0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t a = in[2 * j], c = in[2 * j + 1];
        out[j] = ptx::pack_e4m3x4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                                  __uint_as_float(c << 16) * inv, __uint_as_float(c & 0xffff0000u) * inv);
      }
      if (dst[u] != nullptr) {
        *reinterpret_cast<uint4*>(dst[u]) = make_uint4(out[0], out[1], out[2], out[3]);
        if (lane == 0) *sdst[u] = __uint_as_float((uint32_t)(127 + se) << 23);
      }
    }
  }
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ ReadParams P) {
  constexpr int E = FP8 ? 16 : 8, L = D / E, PER = kThreads / L;
  ptx::grid_dependency_wait();
  const int nv = 2 * P.c.heads_kv;
  const int64_t total = (int64_t)P.total_k * nv;
  const int64_t first = (int64_t)blockIdx.x * (PER * kBatch);
  const int lane = threadIdx.x % L;
  const int b0 = find_sequence(P.cu_k, P.batch, first / nv);
  uint4 x[kBatch];
  float scale[kBatch];
  uint8_t* dst[kBatch];
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    dst[u] = nullptr;
    const int64_t id = first + u * PER + threadIdx.x / L;
    if (id >= total) continue;
    const int64_t t = id / nv;
    const int w = (int)(id - t * nv);
    const bool is_v = w >= P.c.heads_kv;
    const int h = is_v ? w - P.c.heads_kv : w;
    int b = b0;
    while (b < P.batch && (int64_t)P.cu_k[b + 1] <= t) ++b;
    if (b >= P.batch) continue;
    const int a = P.cu_k[b], pos = (int)(t - a);
    // offsets that are out of order (or below zero) leave a row in front of
    // its sequence's start, or past what the table can hold
    if (a < 0 || pos < 0 || (pos >> P.c.page_shift) >= P.c.max_pages) {
      record_bad_cache(P.ws, b);
      continue;
    }
    const int page = __ldg(P.c.table + (int64_t)b * P.c.table_stride + (pos >> P.c.page_shift));
    if ((unsigned)page >= (unsigned)P.c.num_pages) {
      record_bad_cache(P.ws, b);
      continue;
    }
    const int slot = pos & ((1 << P.c.page_shift) - 1);
    const uint8_t* src = (is_v ? P.c.v + page * P.c.v_page + slot * P.c.v_tok + h * P.c.v_head
                               : P.c.k + page * P.c.k_page + slot * P.c.k_tok + h * P.c.k_head) + lane * 16;
    x[u] = __ldcs(reinterpret_cast<const uint4*>(src));
    if constexpr (FP8)
      scale[u] = __ldg((is_v ? P.c.v_scale : P.c.k_scale) +
                       ((((int64_t)page * P.c.heads_kv + h) << P.c.page_shift) + slot));
    dst[u] = (is_v ? P.v + t * P.v_t + h * P.v_h : P.k + t * P.k_t + h * P.k_h) + lane * (E * 2);
  }
#pragma unroll
  for (int u = 0; u < kBatch; ++u) {
    if (dst[u] == nullptr) continue;
    if constexpr (!FP8) {
      *reinterpret_cast<uint4*>(dst[u]) = x[u];
    } else {
      const uint32_t in[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
      uint32_t out[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 lo, hi;
        ptx::e4m3x2_to_float2(in[j] & 0xffffu, lo.x, lo.y);
        ptx::e4m3x2_to_float2(in[j] >> 16, hi.x, hi.y);
        out[2 * j] = ptx::pack_bf16(lo.x * scale[u], lo.y * scale[u]);
        out[2 * j + 1] = ptx::pack_bf16(hi.x * scale[u], hi.y * scale[u]);
      }
      uint4* d = reinterpret_cast<uint4*>(dst[u]);
      d[0] = make_uint4(out[0], out[1], out[2], out[3]);
      d[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

template <class K, class P>
cudaError_t launch(K kern, const P& p, int64_t vectors, int per_block, cudaStream_t stream) {
  const int64_t blocks = (vectors + per_block - 1) / per_block;
  if (blocks <= 0) return cudaSuccess;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  return launch_dependent(kern, p, dim3((unsigned)blocks), kThreads, 0, stream);
}

constexpr int per_block(int d, bool fp8) { return kThreads / (d / (fp8 ? 16 : 8)) * kBatch; }

}  // namespace

cudaError_t cache_append_launch(const AppendParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  const int64_t n = p.tokens * 2 * p.c.heads_kv;
  const int pb = per_block(head_dim, fp8);
  if (head_dim == 128)
    return fp8 ? launch(cache_append_kernel<128, true>, p, n, pb, stream)
               : launch(cache_append_kernel<128, false>, p, n, pb, stream);
  return fp8 ? launch(cache_append_kernel<64, true>, p, n, pb, stream)
             : launch(cache_append_kernel<64, false>, p, n, pb, stream);
}

cudaError_t cache_read_launch(const ReadParams& p, int head_dim, bool fp8, cudaStream_t stream) {
  const int64_t n = (int64_t)p.total_k * 2 * p.c.heads_kv;
  const int pb = per_block(head_dim, fp8);
  if (head_dim == 128)
    return fp8 ? launch(cache_read_kernel<128, true>, p, n, pb, stream)
               : launch(cache_read_kernel<128, false>, p, n, pb, stream);
  return fp8 ? launch(cache_read_kernel<64, true>, p, n, pb, stream)
             : launch(cache_read_kernel<64, false>, p, n, pb, stream);
}

}  // namespace af
