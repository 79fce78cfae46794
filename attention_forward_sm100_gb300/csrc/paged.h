// Declarations shared by the paged-cache kernels and their host API.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn_paged.h"
#include "internal.h"

namespace af {

// Keys per work unit of the streaming attention kernel: 16 per warp and step
// for 256-byte cache rows, 32 for shorter ones (the fixed work of a step then
// weighs half); a group of several warps shares its keys.
constexpr int stream_tile(int row_bytes, int group_warps) { return group_warps == 1 && row_bytes < 256 ? 128 : 64; }
// CTAs of it per SM. A third one hides the latencies of e4m3 at D = 64 (16 sequences
// of up to 32768 keys, GQA 32/8: 69.6 -> 64.2 us; a fourth leaves too few registers,
// 77.6); where two already wait for HBM it does not pay (e4m3, D = 128: 104 -> 118 with
// the half tiles that it needs).
constexpr int stream_ctas(int row_bytes, int row_tile) { return row_bytes == 64 && row_tile == 8 ? 3 : 2; }
constexpr int kMinPage = 16;         // smallest page: one warp's step of keys lies in one page

// The new rows of each sequence (fixed: b * seqlen_q; packed: cu_q) and the
// cached lengths.
struct NewRows {
  const int32_t* cu_q;       // NULL when fixed
  const int32_t* seqlens_k;
  int32_t batch, seqlen_q, total_q, max_k;
};

struct AppendParams {
  CacheView c;
  NewRows s;
  const uint8_t* k;
  const uint8_t* v;
  int64_t k_b, k_t, k_h, v_b, v_t, v_h;   // bytes
  int64_t tokens;
  int32_t wide;                           // 1: k, v and their strides are multiples of 32 bytes
  int32_t block_tokens;                   // set by the launch, as `magic`
  uint32_t magic;
  uint32_t* ws;
};

struct ReadParams {
  CacheView c;
  const int32_t* cu_k;
  uint8_t* k;
  uint8_t* v;
  int64_t k_t, k_h, v_t, v_h;   // bytes
  int32_t batch, total_k;
  int32_t wide;                // as in AppendParams
  int32_t block_tokens;
  uint32_t magic;
  uint32_t* ws;
};

// Widening an e4m3 cache into bf16 pages of kBlockN tokens, [batch * pages][Hkv][kBlockN][D],
// sequence b's in order from page b * pages on, and the block table that says so.
struct WidenParams {
  CacheView c;
  const int32_t* seqlens_k;
  int32_t max_k, batch, pages;
  uint8_t* k;
  uint8_t* v;
  int32_t* table;
  int32_t block_tokens;
  uint32_t magic;
  uint32_t* ws;
};

struct StreamParams {
  CacheView c;
  NewRows s;
  const uint8_t* q;
  int64_t q_b, q_t, q_h;     // bytes
  uint16_t* o;
  float* lse;
  int64_t o_b, o_t, o_h;     // elements
  int32_t heads_q, group, causal;
  int32_t team, team_heads;  // CTAs of a team (the grid is a multiple), KV heads of a member
  int32_t split;             // 1: units are key tiles, segments may span CTAs; 0: units are segments
  float scale_log2;
  uint32_t* ws;
  uint32_t* counters;        // [3 * grid], zero between calls
  float2* part_ml;           // [2 * grid][rows]: running maximum (log2 units) and sum
  float* part_o;             // [2 * grid][rows][D], not normalised
};

// Arguments of the plan and merge kernels of a paged problem on the tcgen05 kernel.
struct PlanParams {
  NewRows s;
  int32_t heads_kv, group, kv_chunk, tokens, causal, ctas;   // as in Tc05Params (tokens = rows_per_tile)
  int32_t pack, pack_tokens, heads_total;
  int32_t max_tiles;         // room in the list
  uint32_t* ws;
  PlanHead* head;
  PlanItem* items;
  PlanPiece* pieces;
  PlanCut* cuts;
  const float* lse_part;     // [slots][256]
  const float* o_part;       // [slots][256][D], normalised
  uint16_t* o;
  float* lse;
  int64_t o_b, o_t, o_h;     // elements
};
cudaError_t paged_plan_launch(const PlanParams& p, cudaStream_t stream);
cudaError_t paged_tile_merge_launch(const PlanParams& p, int head_dim, int max_cut, cudaStream_t stream);

cudaError_t cache_append_launch(const AppendParams& p, int head_dim, bool fp8, cudaStream_t stream);
cudaError_t cache_widen_launch(const WidenParams& p, int head_dim, cudaStream_t stream);
cudaError_t cache_read_launch(const ReadParams& p, int head_dim, bool fp8, cudaStream_t stream);
// Streaming attention over `grid` CTAs with row tiles of 8, 16 or 32 rows.
cudaError_t paged_stream_launch(const StreamParams& p, int head_dim, bool fp8, int row_tile, int grid,
                                cudaStream_t stream);

#ifdef __CUDACC__
// Records the first invalid length, offset or page of a call.
__device__ __forceinline__ void record_bad_cache(uint32_t* ws, int b) {
  if (atomicCAS(&ws[kWsErrorCode], 0u, (uint32_t)kDevErrBadCache) == 0u) atomicExch(&ws[kWsErrorInfo], (uint32_t)b);
}

struct SeqRows {
  int lq, lk, q0;   // new rows, cached keys, first row (packed) or 0
};

struct SeqRaw {
  int lk, a, e;     // as the tensors have them: cached keys, row offsets (packed)
};
__device__ __forceinline__ SeqRaw load_seq_raw(const NewRows& s, int b) {
  SeqRaw w = {s.seqlens_k[b], 0, 0};
  if (s.cu_q != nullptr) {
    w.a = s.cu_q[b];
    w.e = s.cu_q[b + 1];
  }
  return w;
}
// Lengths of sequence b; out of range ones are recorded and cut to what the
// tensors hold.
__device__ __forceinline__ SeqRows checked_seq(const NewRows& s, const SeqRaw& w, int b, uint32_t* ws) {
  SeqRows r;
  r.lk = w.lk;
  r.lq = s.seqlen_q;
  r.q0 = 0;
  bool bad = r.lk < 0 || r.lk > s.max_k;
  if (bad) r.lk = r.lk < 0 ? 0 : s.max_k;
  if (s.cu_q != nullptr) {
    const int a = w.a, e = w.e;
    r.q0 = a;
    r.lq = e - a;
    if (a < 0 || e < a || e > s.total_q) {
      bad = true;
      r.q0 = r.lq = 0;
    } else if (r.lq > s.seqlen_q) {
      bad = true;
      r.lq = s.seqlen_q;
    }
  }
  if (bad) record_bad_cache(ws, b);
  return r;
}
__device__ __forceinline__ SeqRows load_seq(const NewRows& s, int b, uint32_t* ws) {
  return checked_seq(s, load_seq_raw(s, b), b, ws);
}

// A page number of sequence b's table row; one outside the cache is recorded
// and replaced by page 0.
__device__ __forceinline__ int checked_page(const CacheView& c, int page, int b, uint32_t* ws) {
  if ((unsigned)page < (unsigned)c.num_pages) return page;
  record_bad_cache(ws, b);
  return 0;
}
// Page of column `col` of sequence b's table row.
__device__ __forceinline__ int load_page(const CacheView& c, int b, int col, uint32_t* ws) {
  return checked_page(c, __ldg(c.table + (int64_t)b * c.table_stride + col), b, ws);
}
#endif

}  // namespace af
