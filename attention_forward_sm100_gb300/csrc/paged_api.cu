// Host side of the C ABI declared in include/attn_paged.h: argument
// validation, launch planning and workspace layout of the paged-cache
// operators.
#include <string.h>

#include "paged.h"
#include "paged_host.h"
#include "schedule.cuh"

namespace {

using af::report_error;

size_t round256(size_t n) { return (n + 255) & ~(size_t)255; }

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

attn_status check_cache(const attn_kv_cache& c) {
  if (c.dtype != ATTN_DTYPE_BF16 && c.dtype != ATTN_DTYPE_FP8_E4M3)
    return report_error(ATTN_ERR_INVALID_ARG, "unknown cache dtype %d", c.dtype);
  if (c.batch < 0 || c.max_pages < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative batch or max_pages");
  if (c.num_pages <= 0 || c.num_heads_kv <= 0)
    return report_error(ATTN_ERR_INVALID_ARG, "the cache needs at least one page and one head");
  if (c.num_heads_kv > 16384) return report_error(ATTN_ERR_UNSUPPORTED, "more than 16384 heads");
  if (c.head_dim != 64 && c.head_dim != 128)
    return report_error(ATTN_ERR_UNSUPPORTED, "head_dim %d: the paged cache supports 64 and 128", c.head_dim);
  if (c.page_size < af::kMinPage || c.page_size > 65536 || (c.page_size & (c.page_size - 1)))
    return report_error(ATTN_ERR_UNSUPPORTED, "page_size %d is not a power of two from %d to 65536", c.page_size,
                        af::kMinPage);
  if ((int64_t)c.max_pages * c.page_size > 0x7fff0000ll)
    return report_error(ATTN_ERR_UNSUPPORTED, "max_pages * page_size is past 2^31");
  if (c.k == nullptr || c.v == nullptr || !aligned(c.k, 16) || !aligned(c.v, 16))
    return report_error(ATTN_ERR_INVALID_ARG, "cache k and v must be non-NULL and 16-byte aligned");
  if (c.batch > 0 && c.max_pages > 0 && (c.block_table == nullptr || !aligned(c.block_table, 4)))
    return report_error(ATTN_ERR_INVALID_ARG, "block_table must be non-NULL and 4-byte aligned");
  if (c.table_stride < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative table_stride");
  const int es = c.dtype == ATTN_DTYPE_FP8_E4M3 ? 1 : 2;
  for (int i = 0; i < 3; ++i) {
    if (c.k_stride[i] < 0 || c.v_stride[i] < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative cache stride");
    if ((c.k_stride[i] * es) % 16 || (c.v_stride[i] * es) % 16)
      return report_error(ATTN_ERR_INVALID_ARG, "cache strides must be multiples of 16 bytes");
  }
  if (c.dtype == ATTN_DTYPE_FP8_E4M3) {
    if (c.k_scale == nullptr || c.v_scale == nullptr || !aligned(c.k_scale, 16) || !aligned(c.v_scale, 16))
      return report_error(ATTN_ERR_INVALID_ARG, "an e4m3 cache needs 16-byte aligned k_scale and v_scale");
  }
  return ATTN_OK;
}

attn_status check_rows(const char* what, const void* p, const int64_t* stride, int first, int n) {
  if (p == nullptr || !aligned(p, 16))
    return report_error(ATTN_ERR_INVALID_ARG, "%s must be non-NULL and 16-byte aligned", what);
  for (int i = first; i < n; ++i)
    if (stride[i] < 0 || (stride[i] * 2) % 16)
      return report_error(ATTN_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes", what);
  return ATTN_OK;
}

// Whether rows at `p` with these strides (of bf16) all start on 32-byte boundaries.
bool wide_rows(const void* p, const int64_t* stride, int first, int n) {
  bool ok = aligned(p, 32);
  for (int i = first; i < n; ++i) ok = ok && (stride[i] * 2) % 32 == 0;
  return ok;
}

attn_status check_offsets(const char* what, const int32_t* p, bool needed) {
  if ((needed && p == nullptr) || !aligned(p, 4))
    return report_error(ATTN_ERR_INVALID_ARG, "%s must be non-NULL and 4-byte aligned", what);
  return ATTN_OK;
}

attn_status check_workspace(const void* ws) {
  if (ws == nullptr || !aligned(ws, 256))
    return report_error(ATTN_ERR_INVALID_ARG, "workspace must be non-NULL and 256-byte aligned");
  return ATTN_OK;
}

af::CacheView view_of(const attn_kv_cache& c) {
  const int es = c.dtype == ATTN_DTYPE_FP8_E4M3 ? 1 : 2;
  af::CacheView v;
  v.k = static_cast<uint8_t*>(c.k);
  v.v = static_cast<uint8_t*>(c.v);
  v.k_scale = c.k_scale;
  v.v_scale = c.v_scale;
  v.table = c.block_table;
  v.k_page = c.k_stride[0] * es;
  v.k_tok = c.k_stride[1] * es;
  v.k_head = c.k_stride[2] * es;
  v.v_page = c.v_stride[0] * es;
  v.v_tok = c.v_stride[1] * es;
  v.v_head = c.v_stride[2] * es;
  v.table_stride = c.table_stride;
  v.num_pages = c.num_pages;
  v.page_shift = 0;
  while ((1 << v.page_shift) < c.page_size) ++v.page_shift;
  v.max_pages = c.max_pages;
  v.heads_kv = c.num_heads_kv;
  return v;
}

attn_status check_append(const attn_cache_append_params* p) {
  if (p == nullptr) return report_error(ATTN_ERR_INVALID_ARG, "params is NULL");
  attn_status st = check_cache(p->cache);
  if (st != ATTN_OK) return st;
  if (p->seqlen_q < 0 || p->total_q < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative size");
  const bool packed = p->cu_seqlens_q != nullptr;
  if (!packed && (int64_t)p->cache.batch * p->seqlen_q > 0x7fffffffll)
    return report_error(ATTN_ERR_UNSUPPORTED, "more than 2^31 new tokens");
  if (p->cache.batch == 0 || (packed ? p->total_q : p->seqlen_q) == 0) return ATTN_OK;
  if ((st = check_rows("k", p->k, p->k_stride, packed ? 1 : 0, 3)) != ATTN_OK) return st;
  if ((st = check_rows("v", p->v, p->v_stride, packed ? 1 : 0, 3)) != ATTN_OK) return st;
  if ((st = check_offsets("seqlens_k", p->seqlens_k, true)) != ATTN_OK) return st;
  if ((st = check_offsets("cu_seqlens_q", p->cu_seqlens_q, false)) != ATTN_OK) return st;
  return check_workspace(p->workspace);
}

attn_status check_read(const attn_cache_read_params* p) {
  if (p == nullptr) return report_error(ATTN_ERR_INVALID_ARG, "params is NULL");
  attn_status st = check_cache(p->cache);
  if (st != ATTN_OK) return st;
  if (p->total_k < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative size");
  if (p->cache.batch == 0 || p->total_k == 0) return ATTN_OK;
  if ((st = check_rows("k", p->k, p->k_stride, 0, 2)) != ATTN_OK) return st;
  if ((st = check_rows("v", p->v, p->v_stride, 0, 2)) != ATTN_OK) return st;
  if ((st = check_offsets("cu_seqlens_k", p->cu_seqlens_k, true)) != ATTN_OK) return st;
  return check_workspace(p->workspace);
}

bool no_rows(const attn_paged_params* p) {
  return p->cache.batch == 0 || (p->cu_seqlens_q != nullptr ? p->total_q : p->seqlen_q) == 0;
}

// Packed rows under a bound of no new tokens may belong to nobody, or the bound is
// wrong, which the device finds out: planned as for one token.
attn_paged_params planned(const attn_paged_params* p) {
  attn_paged_params q = *p;
  if (q.cu_seqlens_q != nullptr && q.seqlen_q == 0) q.seqlen_q = 1;
  return q;
}

// Everything but the workspace.
attn_status check_paged(const attn_paged_params* p) {
  if (p == nullptr) return report_error(ATTN_ERR_INVALID_ARG, "params is NULL");
  attn_status st = check_cache(p->cache);
  if (st != ATTN_OK) return st;
  const attn_kv_cache& c = p->cache;
  if (p->seqlen_q < 0 || p->seqlen_k < 0 || p->total_q < 0) return report_error(ATTN_ERR_INVALID_ARG, "negative size");
  if (p->num_heads_q <= 0 || p->num_heads_q % c.num_heads_kv)
    return report_error(ATTN_ERR_INVALID_ARG, "num_heads_q %d is not a positive multiple of num_heads_kv %d",
                        p->num_heads_q, c.num_heads_kv);
  if (!(p->softmax_scale > 0.f)) return report_error(ATTN_ERR_INVALID_ARG, "softmax_scale must be a positive number");
  if (p->seqlen_k > (int64_t)c.max_pages * c.page_size)
    return report_error(ATTN_ERR_INVALID_ARG, "seqlen_k %d is past max_pages * page_size", p->seqlen_k);
  if (no_rows(p)) return ATTN_OK;
  const bool packed = p->cu_seqlens_q != nullptr;
  if ((st = check_rows("q", p->q, p->q_stride, packed ? 1 : 0, 3)) != ATTN_OK) return st;
  if ((st = check_rows("o", p->o, p->o_stride, packed ? 1 : 0, 3)) != ATTN_OK) return st;
  if ((st = check_offsets("seqlens_k", p->seqlens_k, true)) != ATTN_OK) return st;
  if ((st = check_offsets("cu_seqlens_q", p->cu_seqlens_q, false)) != ATTN_OK) return st;
  if (!aligned(p->lse, 4)) return report_error(ATTN_ERR_INVALID_ARG, "lse must be 4-byte aligned");
  return ATTN_OK;
}

// The zeroed head of the workspace: the words every kernel of the library uses,
// then the streaming kernel's counters, three per CTA.
constexpr size_t kZeroedBytes = ATTN_PAGED_ZEROED_BYTES;
constexpr int64_t kMaxStreamCtas = (kZeroedBytes - ATTN_FWD_WORKSPACE_BYTES) / 12;

// Two kernels. R = Lq * Hq / Hkv rows share the keys of a (sequence, KV head).
// The streaming kernel reads the cache at close to the copy bandwidth, but its
// work grows with R; the tcgen05 kernel computes 256-row tiles, mostly padding
// while R is small. Measured on both (us, streaming / tcgen05; 64 sequences of up
// to 8192 keys in bf16, 16 of up to 32768 in e4m3, GQA 32/8, d128):
//   R      4          16         32         48         64         128
//   bf16   171 / 218  179 / 220  192 / 220  350 / 222  356 / 224  686 / 228
//   e4m3   106 / 323  117 / 332  201 / 335  371 / 341  373 / 343  731 / 351
constexpr int kStreamRows = 32;
int64_t shared_rows(const attn_paged_params* p) {
  return (int64_t)p->seqlen_q * (p->num_heads_q / p->cache.num_heads_kv);
}
bool use_tc05(const attn_paged_params* p) { return shared_rows(p) > kStreamRows; }

// tcgen05 kernel: query heads packed into a 128-row tile (the largest divisor of
// the group up to 128), tokens of such a tile and of a work tile of two, and the work
// list's memory. Without a list (few keys, where nothing is worth cutting, or
// so many tiles that their whole number per CTA does not matter) every tile is
// taken whole.
struct TilePlan {
  int pack, pack_tokens;
  int tokens;
  int64_t work;      // upper bound of the work tiles
  bool list;
  int max_cut, max_pieces;
  size_t items, pieces, cuts, lse, o;   // bytes, in this order behind the plan's head
  size_t bytes;
};
TilePlan plan_tiles(const attn_paged_params* p) {
  TilePlan t = {};
  const attn_kv_cache& c = p->cache;
  const int group = p->num_heads_q / c.num_heads_kv;
  t.pack = group < af::kBlockM ? group : af::kBlockM;
  while (group % t.pack) --t.pack;
  t.pack_tokens = af::kBlockM / t.pack;
  t.tokens = 2 * t.pack_tokens;
  int64_t token_tiles = (int64_t)c.batch * af::tiles_for(p->seqlen_q, t.tokens);
  if (p->cu_seqlens_q != nullptr && p->total_q / t.tokens + c.batch < token_tiles)
    token_tiles = p->total_q / t.tokens + c.batch;
  t.work = token_tiles * (p->num_heads_q / t.pack);
  t.list = af::tiles_for(p->seqlen_k, af::kBlockN) > af::kListTiles && t.work <= af::kPlanMaxTiles &&
           c.batch <= af::kPlanMaxBatch;
  if (t.list) {
    const int64_t ctas = af::sm_count();
    t.max_cut = (int)(t.work < 2 * ctas ? t.work : 2 * ctas);
    t.max_pieces = (int)(2 * ctas);
    const int64_t slots = t.max_cut + t.max_pieces;
    t.items = round256((size_t)(t.work + slots) * sizeof(af::PlanItem));
    t.pieces = round256((size_t)t.max_pieces * sizeof(af::PlanPiece));
    t.cuts = round256((size_t)t.max_cut * sizeof(af::PlanCut));
    t.lse = round256((size_t)slots * af::kRowsPerTile * sizeof(float));
    t.o = (size_t)slots * af::kRowsPerTile * c.head_dim * sizeof(float);
    t.bytes = 256 + t.items + t.pieces + t.cuts + t.lse + t.o;
  }
  return t;
}

struct StreamPlan {
  int row_tile;
  int split;
  int team;            // CTAs that walk together, each with its own heads
  int64_t grid;
  int64_t units;       // upper bound of the work units
  size_t ml_bytes, o_bytes;
};

// Row tiles of 8, 16 or 32 rows, the smallest that holds a sequence's rows; two
// or three CTAs per SM. Segments of up to kUnsplitTiles key tiles are not cut: the
// join would cost more than the longer CTA. Nor are those of up to kUnsplitKeys
// keys if they are at least a quarter as many as the CTAs and at most twice.
// GQA 32/8, d128, us cut / whole: 12 sequences of up to 300 keys, bf16: 12.8 / 7.0;
// 32 sequences of up to 1000 keys, bf16 22.7 / 17.5, e4m3 21.2 / 14.9; 8 of them
// 13.7 / 13.6; 75 of them 36.7 / 34.6; but 3 of them 9.1 / 12.3, 256 of them 94 / 112.
// Where the bound on the lengths allows more key tiles than the device counts (in
// 32 bits), segments, which are then thousands, are left whole too.
constexpr int kUnsplitTiles = 4;
constexpr int kUnsplitKeys = 1024;
constexpr int64_t kMaxUnits = 0x3fffffff;
// Of cut segments, the CTAs of a team take different heads of the same keys, so
// that what HBM is asked for at one time lies together; unteamed, CTAs read
// strided rows of one head each. The team is the largest divisor of Hkv up to 16
// (more would leave more of the grid's remainder idle). us, unteamed / team of 4 /
// of 16 at most: 64 sequences of up to 8192 keys, GQA 32/8, d128 bf16: 182 / 174 / 171;
// 16 of up to 32768 e4m3: 125 / 109 / 106, with d64 88 / 76 / 74; with 32, 13, 11 KV
// heads 123, 188, 163 / - / 106, 172, 146; head-major pages, d128 bf16 and e4m3:
// 179, 110 / - / 171, 105.
constexpr int kMaxTeam = 16;
StreamPlan plan_stream(const attn_paged_params* p) {
  StreamPlan s = {};
  const int64_t rows = shared_rows(p);
  s.row_tile = rows <= 8 ? 8 : (rows <= 16 ? 16 : 32);
  const int64_t rt = s.row_tile;
  const int row_bytes = p->cache.head_dim * (p->cache.dtype == ATTN_DTYPE_FP8_E4M3 ? 1 : 2);
  const int64_t segments = (int64_t)p->cache.batch * p->cache.num_heads_kv * ((rows + rt - 1) / rt);
  const int64_t tiles = af::tiles_for(p->seqlen_k, af::stream_tile(row_bytes, s.row_tile <= 16 ? 1 : s.row_tile / 16));
  const int64_t ctas = (int64_t)af::stream_ctas(row_bytes, s.row_tile) * af::sm_count();
  const bool one_wave = 4 * segments >= ctas && segments <= 2 * ctas;
  s.split = tiles > kUnsplitTiles && !(one_wave && p->seqlen_k <= kUnsplitKeys) && segments <= kMaxUnits / tiles ? 1 : 0;
  s.units = segments * (s.split ? tiles : 1);
  const int64_t most = ctas < kMaxStreamCtas ? ctas : kMaxStreamCtas;
  s.grid = s.units < most ? s.units : most;
  s.team = 1;
  if (s.split) {
    const int heads = p->cache.num_heads_kv;
    s.team = heads < kMaxTeam ? heads : kMaxTeam;
    while (heads % s.team) --s.team;
    s.grid -= s.grid % s.team;
  }
  if (s.split) {
    s.ml_bytes = round256((size_t)(2 * s.grid * rt) * sizeof(float2));
    s.o_bytes = (size_t)(2 * s.grid * rt) * p->cache.head_dim * sizeof(float);
  }
  return s;
}

// Whether an e4m3 cache is widened to bf16 pages in scratch memory first, for the
// tcgen05 kernel's bf16 form to read: that costs K and V once each way, the e4m3
// form extra work for every 256 rows. us, widened / e4m3 form, GQA 32/8, d128,
// 32768 keys: 64 new tokens (R = 256) 79 / 77, 128: 100 / 104, 256: 143 / 157,
// 512: 230 / 265, 2048: 711 / 897; four ragged sequences of up to 12000 keys and 1023
// new tokens 372 / 468, d64 316 / 422; with 32 KV heads 485 / 480, of up to 512 new
// tokens (R about 300 on average) 386 / 342. Not where the scratch memory would
// pass kWidenBytes. K is rounded to bf16 with it (D = 128: without it not), which
// scales that are powers of two do not notice.
constexpr int64_t kWidenRows = 512, kWidenBytes = 1ll << 30;
struct WidenPlan {
  bool on;
  int pages;                 // of kBlockN tokens, per sequence
  size_t table, rows;        // bytes: block table, K (and V as many)
};
WidenPlan plan_widen(const attn_paged_params* p) {
  WidenPlan w = {};
  const attn_kv_cache& c = p->cache;
  if (c.dtype != ATTN_DTYPE_FP8_E4M3 || !use_tc05(p)) return w;
  const int64_t tokens = p->cu_seqlens_q != nullptr ? p->total_q : (int64_t)c.batch * p->seqlen_q;
  w.pages = af::tiles_for(p->seqlen_k, af::kBlockN);
  const int64_t n = (int64_t)c.batch * w.pages, row = (int64_t)c.num_heads_kv * af::kBlockN * c.head_dim * 2;
  w.on = w.pages > 0 && tokens * (p->num_heads_q / c.num_heads_kv) >= kWidenRows * c.batch &&
         n <= kWidenBytes / (2 * row);
  if (!w.on) return w;
  w.table = round256((size_t)n * sizeof(int32_t));
  w.rows = (size_t)(n * row);
  return w;
}

// Bytes behind the zeroed head.
size_t scratch_need(const attn_paged_params* p) {
  if (use_tc05(p)) {
    const WidenPlan w = plan_widen(p);
    return round256(plan_tiles(p).bytes) + w.table + 2 * w.rows;
  }
  const StreamPlan s = plan_stream(p);
  return s.ml_bytes + s.o_bytes;
}

// Stride of a dimension of size 1 (never used, but a tensor map wants a legal one).
int64_t legal(int64_t stride, int64_t size) { return size > 1 ? stride : 16; }

attn_status launch_tiles(const attn_paged_params* p, uint8_t* scratch, cudaStream_t stream) {
  const TilePlan plan = plan_tiles(p);
  attn_kv_cache c = p->cache;
  const bool packed = p->cu_seqlens_q != nullptr;
  if (const WidenPlan w = plan_widen(p); w.on) {
    af::WidenParams wp;
    memset(&wp, 0, sizeof(wp));
    uint8_t* at = scratch + round256(plan.bytes);
    wp.c = view_of(c);
    wp.seqlens_k = p->seqlens_k;
    wp.max_k = p->seqlen_k;
    wp.batch = c.batch;
    wp.pages = w.pages;
    wp.table = reinterpret_cast<int32_t*>(at);
    wp.k = at + w.table;
    wp.v = wp.k + w.rows;
    wp.ws = static_cast<uint32_t*>(p->workspace);
    const cudaError_t e = af::cache_widen_launch(wp, c.head_dim, stream);
    if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "cache widening launch failed: %s", cudaGetErrorString(e));
    c.k = wp.k;
    c.v = wp.v;
    c.k_scale = c.v_scale = nullptr;
    c.block_table = wp.table;
    c.dtype = ATTN_DTYPE_BF16;
    c.page_size = af::kBlockN;
    c.num_pages = c.batch * w.pages;
    c.max_pages = w.pages;
    c.table_stride = w.pages;
    for (int64_t* s : {c.k_stride, c.v_stride}) {
      s[0] = (int64_t)c.num_heads_kv * af::kBlockN * c.head_dim;
      s[1] = c.head_dim;
      s[2] = (int64_t)af::kBlockN * c.head_dim;
    }
  }
  af::Tc05Params prm;
  memset(&prm, 0, sizeof(prm));
  const CUtensorMapDataType bf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int64_t q_tokens = packed ? p->total_q : p->seqlen_q, q_batches = packed ? 1 : c.batch;
  const int page_rows = c.page_size < af::kBlockN ? c.page_size : af::kBlockN;
  attn_status st = af::encode_map(
      &prm.tm_q, bf16, p->q, {c.head_dim, p->num_heads_q, q_tokens, q_batches},
      {legal(p->q_stride[2] * 2, p->num_heads_q), legal(p->q_stride[1] * 2, q_tokens), legal(p->q_stride[0] * 2, q_batches)},
      {64, plan.pack, plan.pack_tokens, 1});
  if (st != ATTN_OK) return st;
  const bool fp8 = c.dtype == ATTN_DTYPE_FP8_E4M3;
  // (of an e4m3 cache only K with D = 128 is read through a map)
  for (int i = 0; i < (fp8 ? (c.head_dim == 128 ? 1 : 0) : 2); ++i) {
    const int64_t* s = i ? c.v_stride : c.k_stride;
    const int64_t es = fp8 ? 1 : 2;
    st = af::encode_map(i ? &prm.tm_v : &prm.tm_k, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : bf16, i ? c.v : c.k,
                        {c.head_dim, c.num_heads_kv, c.page_size, c.num_pages},
                        {legal(s[2] * es, c.num_heads_kv), s[1] * es, legal(s[0] * es, c.num_pages)},
                        {fp8 ? 128 : 64, 1, page_rows, 1});
    if (st != ATTN_OK) return st;
  }
  prm.q = static_cast<const uint8_t*>(p->q);
  prm.q_b = packed ? 0 : p->q_stride[0] * 2;
  prm.q_t = p->q_stride[1] * 2;
  prm.q_h = p->q_stride[2] * 2;
  prm.cu_q = p->cu_seqlens_q;
  prm.o = static_cast<uint16_t*>(p->o);
  prm.lse = p->lse;
  prm.ws = static_cast<uint32_t*>(p->workspace);
  prm.o_stride_b = packed ? 0 : p->o_stride[0];
  prm.o_stride_t = p->o_stride[1];
  prm.o_stride_h = p->o_stride[2];
  prm.o_store32 = aligned(p->o, 32) && (p->o_stride[2] * 2) % 32 == 0 && (p->o_stride[1] * 2) % 32 == 0 &&
                  (packed || (p->o_stride[0] * 2) % 32 == 0);
  prm.batch = c.batch;
  prm.seqlen_q = p->seqlen_q;
  prm.seqlen_k = p->seqlen_k;
  prm.heads_q = p->num_heads_q / plan.pack;
  prm.heads_kv = c.num_heads_kv;
  prm.group = prm.heads_q / c.num_heads_kv;
  prm.rows_per_tile = plan.tokens;
  prm.tiles_per_seq = af::tiles_for(p->seqlen_q, plan.tokens);
  prm.kv_chunk = af::choose_kv_chunk(p->seqlen_k, (fp8 ? 2ll : 4ll) * c.head_dim, c.num_heads_kv, af::kL2ChunkBudget);
  prm.packed = packed ? 1 : 0;
  prm.total_q = packed ? p->total_q : 0;
  prm.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  prm.timeout_ns = 2000000000ull;
  prm.schedule = ATTN_SCHEDULE_DYNAMIC;
  prm.num_splits = 1;
  prm.cache = view_of(c);
  prm.seqlens_k = p->seqlens_k;
  prm.max_k = p->seqlen_k;
  prm.pack = plan.pack;
  prm.pack_tokens = plan.pack_tokens;
  prm.heads_total = p->num_heads_q;
  const int sms = af::sm_count();
  const int64_t most = plan.list ? plan.work + plan.max_pieces : plan.work;
  const int grid = (int)(most < sms ? most : sms);
  // A full grid gains nothing from starting before the kernel in front of it
  // ends, but for the plan kernel, which is one block.
  prm.dependent_launch = plan.list || grid < sms ? 1 : 0;
  af::PlanParams pp;
  memset(&pp, 0, sizeof(pp));
  cudaError_t e = cudaSuccess;
  if (plan.list) {
    uint8_t* ws = scratch;
    pp.s = {p->cu_seqlens_q, p->seqlens_k, c.batch, p->seqlen_q, p->total_q, p->seqlen_k};
    pp.heads_kv = c.num_heads_kv;
    pp.group = prm.group;
    pp.kv_chunk = prm.kv_chunk;
    pp.tokens = plan.tokens;
    pp.causal = p->causal != 0;
    pp.ctas = grid;
    pp.pack = plan.pack;
    pp.pack_tokens = plan.pack_tokens;
    pp.heads_total = p->num_heads_q;
    pp.max_tiles = (int32_t)plan.work;
    pp.ws = prm.ws;
    pp.head = reinterpret_cast<af::PlanHead*>(ws);
    pp.items = reinterpret_cast<af::PlanItem*>(ws += 256);
    pp.pieces = reinterpret_cast<af::PlanPiece*>(ws += plan.items);
    pp.cuts = reinterpret_cast<af::PlanCut*>(ws += plan.pieces);
    prm.lse_part = reinterpret_cast<float*>(ws += plan.cuts);
    prm.o_part = reinterpret_cast<float*>(ws += plan.lse);
    pp.lse_part = prm.lse_part;
    pp.o_part = prm.o_part;
    pp.o = prm.o;
    pp.lse = p->lse;
    pp.o_b = prm.o_stride_b;
    pp.o_t = prm.o_stride_t;
    pp.o_h = prm.o_stride_h;
    prm.plan = pp.head;
    prm.items = pp.items;
    prm.pieces = pp.pieces;
    e = af::paged_plan_launch(pp, stream);
    if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "paged plan launch failed: %s", cudaGetErrorString(e));
  }
  const int mask = (p->causal ? af::kMaskCausal : 0) | (plan.list ? af::kMaskNoneSplit : 0);
  const int variant = c.head_dim == 64 ? (fp8 ? af::kVarPaged8D64 : af::kVarPagedD64)
                                       : (fp8 ? af::kVarPaged8D128 : af::kVarPagedD128);
  e = af::tc05_launch(variant, mask, prm, grid, stream);
  if (e == cudaSuccess && plan.list) e = af::paged_tile_merge_launch(pp, c.head_dim, plan.max_cut, stream);
  if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "paged attention launch failed: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

}  // namespace

attn_status af::paged_fwd(const attn_paged_params* params, void* scratch, size_t scratch_bytes, cudaStream_t stream) {
  report_error(ATTN_OK, "%s", "");
  attn_status st = check_paged(params);
  if (st != ATTN_OK) return st;
  if (no_rows(params)) return ATTN_OK;
  const attn_paged_params with_rows = planned(params), *p = &with_rows;
  if ((st = check_workspace(p->workspace)) != ATTN_OK) return st;
  const size_t need = scratch_need(p);
  if (p->workspace_bytes < kZeroedBytes + (scratch != nullptr ? 0 : need))
    return report_error(ATTN_ERR_INVALID_ARG, "workspace of at least %zu bytes is required", kZeroedBytes + need);
  if (scratch != nullptr && (scratch_bytes < need || !aligned(scratch, 256)))
    return report_error(ATTN_ERR_INVALID_ARG, "scratch memory of at least %zu bytes is required", need);
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  uint8_t* const room = scratch != nullptr ? static_cast<uint8_t*>(scratch) : ws + kZeroedBytes;
  if (use_tc05(p)) return launch_tiles(p, room, stream);
  const StreamPlan plan = plan_stream(p);
  if (plan.units > kMaxUnits) return report_error(ATTN_ERR_UNSUPPORTED, "more than 2^30 sequences times KV heads");
  const bool packed = p->cu_seqlens_q != nullptr;
  af::StreamParams a;
  memset(&a, 0, sizeof(a));
  a.c = view_of(p->cache);
  a.s.cu_q = p->cu_seqlens_q;
  a.s.seqlens_k = p->seqlens_k;
  a.s.batch = p->cache.batch;
  a.s.seqlen_q = p->seqlen_q;
  a.s.total_q = p->total_q;
  a.s.max_k = p->seqlen_k;
  a.q = static_cast<const uint8_t*>(p->q);
  a.q_b = packed ? 0 : p->q_stride[0] * 2;
  a.q_t = p->q_stride[1] * 2;
  a.q_h = p->q_stride[2] * 2;
  a.o = static_cast<uint16_t*>(p->o);
  a.o_b = packed ? 0 : p->o_stride[0];
  a.o_t = p->o_stride[1];
  a.o_h = p->o_stride[2];
  a.lse = p->lse;
  a.heads_q = p->num_heads_q;
  a.group = p->num_heads_q / p->cache.num_heads_kv;
  a.causal = p->causal != 0;
  a.team = plan.team;
  a.team_heads = p->cache.num_heads_kv / plan.team;
  a.split = plan.split;
  a.scale_log2 = p->softmax_scale * 1.4426950408889634f;
  a.ws = reinterpret_cast<uint32_t*>(ws);
  a.counters = reinterpret_cast<uint32_t*>(ws + ATTN_FWD_WORKSPACE_BYTES);
  a.part_ml = reinterpret_cast<float2*>(room);
  a.part_o = reinterpret_cast<float*>(room + plan.ml_bytes);
  const cudaError_t e =
      af::paged_stream_launch(a, p->cache.head_dim, p->cache.dtype == ATTN_DTYPE_FP8_E4M3, plan.row_tile,
                              (int)plan.grid, stream);
  if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "paged attention launch failed: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

extern "C" {

size_t attn_paged_params_size(int32_t which) {
  switch (which) {
    case 0: return sizeof(attn_cache_append_params);
    case 1: return sizeof(attn_cache_read_params);
    case 2: return sizeof(attn_paged_params);
  }
  return 0;
}

attn_status attn_cache_append(const attn_cache_append_params* p, attn_stream_t stream) {
  report_error(ATTN_OK, "%s", "");
  const attn_status st = check_append(p);
  if (st != ATTN_OK) return st;
  const bool packed = p->cu_seqlens_q != nullptr;
  if (p->cache.batch == 0 || (packed ? p->total_q : p->seqlen_q) == 0) return ATTN_OK;
  af::AppendParams a;
  memset(&a, 0, sizeof(a));
  a.c = view_of(p->cache);
  a.s.cu_q = p->cu_seqlens_q;
  a.s.seqlens_k = p->seqlens_k;
  a.s.batch = p->cache.batch;
  a.s.seqlen_q = p->seqlen_q;
  a.s.total_q = p->total_q;
  a.s.max_k = p->cache.max_pages * p->cache.page_size;
  a.k = static_cast<const uint8_t*>(p->k);
  a.v = static_cast<const uint8_t*>(p->v);
  a.k_b = packed ? 0 : p->k_stride[0] * 2;
  a.k_t = p->k_stride[1] * 2;
  a.k_h = p->k_stride[2] * 2;
  a.v_b = packed ? 0 : p->v_stride[0] * 2;
  a.v_t = p->v_stride[1] * 2;
  a.v_h = p->v_stride[2] * 2;
  a.wide = wide_rows(p->k, p->k_stride, packed ? 1 : 0, 3) && wide_rows(p->v, p->v_stride, packed ? 1 : 0, 3);
  a.tokens = packed ? p->total_q : (int64_t)p->cache.batch * p->seqlen_q;
  a.ws = static_cast<uint32_t*>(p->workspace);
  const cudaError_t e = af::cache_append_launch(a, p->cache.head_dim, p->cache.dtype == ATTN_DTYPE_FP8_E4M3,
                                                reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "cache append launch failed: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

attn_status attn_cache_read(const attn_cache_read_params* p, attn_stream_t stream) {
  report_error(ATTN_OK, "%s", "");
  const attn_status st = check_read(p);
  if (st != ATTN_OK) return st;
  if (p->cache.batch == 0 || p->total_k == 0) return ATTN_OK;
  af::ReadParams r;
  memset(&r, 0, sizeof(r));
  r.c = view_of(p->cache);
  r.cu_k = p->cu_seqlens_k;
  r.k = static_cast<uint8_t*>(p->k);
  r.v = static_cast<uint8_t*>(p->v);
  r.k_t = p->k_stride[0] * 2;
  r.k_h = p->k_stride[1] * 2;
  r.v_t = p->v_stride[0] * 2;
  r.v_h = p->v_stride[1] * 2;
  r.wide = wide_rows(p->k, p->k_stride, 0, 2) && wide_rows(p->v, p->v_stride, 0, 2);
  r.batch = p->cache.batch;
  r.total_k = p->total_k;
  r.ws = static_cast<uint32_t*>(p->workspace);
  const cudaError_t e = af::cache_read_launch(r, p->cache.head_dim, p->cache.dtype == ATTN_DTYPE_FP8_E4M3,
                                              reinterpret_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return report_error(ATTN_ERR_CUDA, "cache read launch failed: %s", cudaGetErrorString(e));
  return ATTN_OK;
}

size_t attn_paged_workspace_bytes(const attn_paged_params* p) {
  if (check_paged(p) != ATTN_OK || no_rows(p)) return kZeroedBytes;
  const attn_paged_params plan = planned(p);
  return kZeroedBytes + scratch_need(&plan);
}

attn_status attn_paged_fwd(const attn_paged_params* p, attn_stream_t stream) {
  return af::paged_fwd(p, nullptr, 0, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
