// Declarations shared by the host API and the kernel translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/attn_fwd.h"

namespace af {

constexpr int kRowsPerTile = 256;   // query rows per work tile of the tcgen05 kernel (one CTA)
constexpr int kRowsPerTilePair = 512;   // the same for a CTA pair (two M = 256 MMA tiles)
constexpr int kBlockM = 128;        // query rows per MMA tile (one TMEM lane per row)
constexpr int kBlockN = 128;        // keys per K/V tile
constexpr int64_t kL2ChunkBudget = 48ll << 20;   // K/V bytes one scheduling chunk may keep in L2
constexpr int64_t kL2ChunkBudgetFp8 = 24ll << 20;   // the same for fp8 Q/K (measured best)
constexpr int kMaxSplits = 64;      // split-KV ranges per query tile (the merge kernel holds 2 per lane)

// Workspace words (uint32 each).
enum WorkspaceWord : int {
  kWsTileCounter = 0,   // next dynamic work index minus gridDim.x
  kWsDoneCounter = 1,   // CTAs finished (the last one resets both counters)
  kWsErrorCode = 2,     // 0 or a device error code
  kWsErrorInfo = 3,     // block, role and barrier of the first error
  kWsCountersLeft = 4,  // 1: a timeout may have left counters behind the words (paged attention) at any value
  kWsWords = 5
};

// Device error codes recorded in kWsErrorCode.
enum DeviceError : uint32_t {
  kDevErrNone = 0,
  kDevErrTimeout = 1,
  kDevErrBadSeqlens = 3,   // packed offsets out of order or past total_q / total_k (info: sequence)
  kDevErrBadCache = 4,     // paged cache: a length, offset or page number out of range (info: sequence)
  kDevErrBadPosition = 5,  // rotary: an offset out of order or a position outside the table (info: sequence, or row)
};

// The cache as the kernels see it; strides in bytes.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* table;
  int64_t k_page, k_tok, k_head;
  int64_t v_page, v_tok, v_head;
  int64_t table_stride;   // elements
  int32_t num_pages, page_shift, max_pages, heads_kv;
};

// Work list of a paged problem (paged_plan.cu): a query tile and the key tiles
// [j0, j1) of it to visit.
struct PlanItem {
  int32_t b, h, t;         // sequence, tile of heads, tile of tokens
  int32_t q_start, lq, lk; // the sequence's first row, new tokens, keys
  int32_t j0, j1;
  int32_t slot;            // partial result to write, or -1: the tile is whole
};
struct PlanPiece {
  int32_t first, last;     // items of one schedule entry
};
struct PlanCut {
  PlanItem item;           // slot: the first part's
  int32_t parts;
};
struct PlanHead {
  int32_t whole, pieces, cut;
  int32_t pad;
};
constexpr int kPlanMaxBatch = 1024;
constexpr int64_t kPlanMaxTiles = 8192;
constexpr int kMinPieceUnits = 4;   // key tiles of a piece worth its set-up and its share of the merge
constexpr int kListTiles = 16;      // up to so many key tiles every query tile is taken whole, without a list

// Everything the tcgen05 kernel needs, passed as one __grid_constant__ struct.
struct Tc05Params {
  CUtensorMap tm_q;        // Q (nope part): box {64 or 128 elements, 1, 128, 1}
  CUtensorMap tm_k;        // K (nope part)
  CUtensorMap tm_v;        // V: box {64, 1, 128, 1}
  CUtensorMap tm_qr;       // Q rope part (rope only)
  CUtensorMap tm_kr;       // K rope part (rope only): box {64, 1, 128, 1}
  const float* q_scale;    // fp8 only
  const float* k_scale;
  const int32_t* cu_q;     // packed only
  const int32_t* cu_k;
  const int32_t* cu_v;     // packed e4m3 V only: key starts of the sequences along V's key dimension
  int32_t total_v;         // packed e4m3 V: length of V's key dimension
  uint16_t* o;             // output rows (bf16 bits)
  float* lse;
  uint32_t* ws;            // workspace words
  int64_t o_stride_b, o_stride_t, o_stride_h;  // elements
  int32_t o_store32;       // 1: o and every row stride are 32-byte aligned (256-bit row stores)
  int32_t batch, seqlen_q, seqlen_k, heads_q, heads_kv, group;
  int32_t tiles_per_seq;   // fixed length: ceil(Sq / rows_per_tile)
  int32_t rows_per_tile;   // query rows per work tile (kRowsPerTile, or kRowsPerTilePair for CTA pairs)
  int32_t kv_chunk;        // KV heads per scheduling chunk
  int64_t total_work;      // fixed length: exact number of work tiles
  int32_t packed;
  int32_t total_q;         // packed: rows of q (LSE and q_scale layout [Hq, Tq])
  int32_t total_k;         // packed: rows of k (k_scale layout [Hkv, Tk])
  float scale_log2;        // softmax_scale * log2(e)
  uint64_t timeout_ns;     // limit of every device wait
  int32_t withhold_v;      // testing: block 0 skips its first V tile load
  int32_t schedule;        // attn_schedule: how the producer advances to its next work index
  int32_t dependent_launch; // host only: launch as a programmatic dependent of the previous kernel
  int32_t num_splits;      // key ranges per query tile (1: no split-KV)
  int32_t kv_tiles;        // split-KV: ceil(seqlen_k / kBlockN)
  float* lse_part;         // split-KV: partial LSE [splits][B][Hq][Sq] / [splits][Hq][Tq]
  float* o_part;           // split-KV: partial O (normalised, fp32) [splits][rows][Hq][Dv]
  // Paged variants only. heads_q then counts tiles of `pack` query heads
  // that share a KV head, group the tiles of one KV head, rows_per_tile the
  // tokens of a work tile; tm_k / tm_v map (depth, head, slot, page).
  CacheView cache;
  const int32_t* seqlens_k;   // [B] cached keys
  int32_t max_k;           // upper bound of them
  int32_t pack;            // query heads in a tile (at most 128)
  int32_t pack_tokens;     // tokens of a 128-row MMA tile, 128 / pack; its rows: token * pack + head
  int32_t heads_total;     // Hq
  const uint8_t* q;        // e4m3 cache: Q itself (split by the kernel), byte strides
  int64_t q_b, q_t, q_h;
  const PlanHead* plan;    // work list, or NULL: every query tile whole, in order
  const PlanItem* items;
  const PlanPiece* pieces;
};

// Arguments of the split-KV merge kernel.
struct SplitCombineParams {
  const float* lse_part;   // [splits][B][Hq][Sq], packed [splits][Hq][Tq]
  const float* o_part;     // [splits][rows][Hq][Dv], rows = B*Sq or Tq
  uint16_t* o;             // bf16 output rows
  float* lse;              // [B][Hq][Sq] / [Hq][Tq], or NULL
  int32_t splits, batch, seqlen_q, heads_q;
  int32_t packed, total_q;
  int64_t o_stride_b, o_stride_t, o_stride_h;   // elements
};

// Kernel variants of the tcgen05 path.
enum Tc05Variant : int {
  kVarD64 = 0,        // bf16, Dqk = Dv = 64
  kVarD128 = 1,       // bf16, Dqk = Dv = 128
  kVarD128Rope64 = 2, // bf16, Dqk = 128 + rope 64, Dv = 128
  kVarFp8D128 = 3,    // fp8 e4m3 Q/K, Dqk = Dv = 128
  kVarFp8QkvD128 = 4, // fp8 e4m3 Q/K/V (depth-major V, P rounded to e4m3), Dqk = Dv = 128
  kVarD128Pair = 5,   // kVarD128 on CTA pairs (M = 256 MMAs over two CTAs)
  kVarD128Rope64Pair = 6, // kVarD128Rope64 on CTA pairs
  kVarPagedD64 = 7,    // bf16 paged cache, D = 64
  kVarPagedD128 = 8,   // bf16 paged cache, D = 128
  kVarPaged8D64 = 9,   // e4m3 paged cache, D = 64
  kVarPaged8D128 = 10, // e4m3 paged cache, D = 128
  kVarCount = 11
};

struct Tc05Config {
  int smem_bytes;
  int k_stages;
  int v_stages;
  int threads;
  int tmem_cols;
};

// Records the calling thread's last-error text (attn_fwd_last_error) and
// returns `st`.
attn_status report_error(attn_status st, const char* fmt, ...);

// 4-D tensor map of a swizzled box (strides of dimensions 1 to 3 in
// bytes); the calling thread's last error says why it failed.
attn_status encode_map(CUtensorMap* map, CUtensorMapDataType type, const void* base, const int64_t (&dims)[4],
                       const int64_t (&strides)[3], const int (&box)[4],
                       CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B);
// SMs of the current device (148 when it cannot be asked).
int sm_count();

// Static configuration of a variant (host).
Tc05Config tc05_config(int variant);
// Flavours of the tcgen05 kernel, two bits: causal mask (1) and split-KV
// (2), so that a kernel carries only the code its calls run (the split
// partial stores, for one, are compiled out of the unsplit flavours). Pair
// variants have no causal split flavour.
enum Tc05Mask : int { kMaskNone = 0, kMaskCausal = 1, kMaskNoneSplit = 2, kMaskCausalSplit = 3 };
// Launch of one variant (defined in the per-variant translation units); a
// pair variant's grid counts CTAs and must be even.
cudaError_t tc05_launch(int variant, int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
// Pair variants: clusters of two CTAs that fit on the current device at once
// (0 when unknown).
int tc05_max_clusters(int variant);
inline bool tc05_is_pair(int variant) { return variant == kVarD128Pair || variant == kVarD128Rope64Pair; }
// Launch of the split-KV merge kernel (head_dim_v 64 or 128).
cudaError_t splitkv_combine_launch(const SplitCombineParams& p, int head_dim_v, cudaStream_t stream);
// Launch of the plain CUDA-core kernel.
cudaError_t simple_launch(const attn_fwd_params& p, cudaStream_t stream);

}  // namespace af
