// The work list of the tcgen05 kernel for a paged problem, and the merge of
// the partial results it leaves.
//
// The lengths are on the device, so the list is made there: one block, before
// the attention kernel (which is launched as its dependent). Query tiles of
// 256 rows are worth as many units as key tiles they see. The W tiles, those
// of the longest sequences first, are handed out whole as long as that fills
// every CTA evenly:
//   whole = floor(W / ctas) * ctas tiles (one CTA-wave fewer when sequences
//   differ, because then so do the tiles of the last full wave);
// the units of the remaining tiles (fewer than two waves) are cut into equal
// pieces, one per CTA (two when sequences differ), without regard to tile
// borders. So every CTA gets the same number of units, and only the tiles that
// a piece border cuts leave partial results: 256 tiles of 256 units on 152 CTAs
// take 2 * 256 units when handed out whole, 449 when each is cut in four (and
// four partial results of everything), 431 + the merge of 104 tiles this way.
// Cutting costs about 8 units (of ~1.5 us: the merge's launch) and one for every
// 18 segments (their set-up and the traffic of the partial results), and is left
// where it evens out less: 384 tiles of four sequences of 3271 to 12000 keys
// take 346 us whole, 369 us cut; 256 tiles of one sequence of 32768 keys 782 us
// whole, 687 us cut.
// Whole tiles keep the order in which CTAs of one KV head run side by side
// over the same keys, which L2 then serves; only the cut ones do not.
//
// A piece is one entry of the dynamic schedule, its segments run one after
// the other in one CTA. Segment (piece p, cut tile i) has index and partial
// slot p + i: unique, because from one segment to the next either p or i grows.
#include <limits.h>
#include <math.h>

#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "schedule.cuh"

namespace af {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kPlanThreads = 1024;
static_assert(kPlanMaxBatch <= kPlanThreads, "one thread per sequence");

// Inclusive sum over the block (all threads).
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += n;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v += warp_sums[warp - 1];
  __syncthreads();
  return v;
}

// The last thread's inclusive sum.
__device__ __forceinline__ int block_total(int incl) {
  __shared__ int total;
  if (threadIdx.x == blockDim.x - 1) total = incl;
  __syncthreads();
  const int t = total;
  __syncthreads();
  return t;
}

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PlanParams P) {
  __shared__ SeqRows seq[kPlanMaxBatch];        // sequences, the longest first
  __shared__ int16_t who[kPlanMaxBatch];        // and their numbers
  __shared__ int ends[kPlanMaxBatch];           // query tiles up to and including each
  __shared__ int key[kPlanMaxBatch];
  __shared__ int sums[32];
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int tid = threadIdx.x, B = P.s.batch;
  SeqRows r = {0, 0, 0};
  if (tid < B) {
    r = load_seq(P.s, tid, P.ws);
    key[tid] = r.lk;
  }
  __syncthreads();
  if (tid < B) {
    int rank = 0;
    for (int b = 0; b < B; ++b) rank += (key[b] > r.lk || (key[b] == r.lk && b < tid)) ? 1 : 0;
    seq[rank] = r;
    who[rank] = (int16_t)tid;
  }
  __syncthreads();
  const int heads = P.heads_kv * P.group;       // tiles of heads
  const int mine = tid < B ? tiles_for(seq[tid].lq, P.tokens) * heads : 0;
  const int end = block_scan(mine, sums);
  if (tid < B) ends[tid] = end;
  __syncthreads();
  int W = B > 0 ? ends[B - 1] : 0;
  if (W > P.max_tiles) {   // overlapping offsets: more rows than there are
    if (tid == 0) record_bad_cache(P.ws, 0);
    W = 0;
  }
  // Tile `x` of the list; returns the key tiles it sees.
  auto tile_at = [&](int x, PlanItem& it) {
    int lo = 0, hi = B - 1;                      // the first sequence with ends > x
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (ends[mid] > x) hi = mid;
      else lo = mid + 1;
    }
    const SeqRows s = seq[lo];
    const int T = tiles_for(s.lq, P.tokens);
    const WorkTile w = decode_in_sequence(x - (lo > 0 ? ends[lo - 1] : 0), who[lo], T, P.group, P.heads_kv, P.kv_chunk);
    const int kv_end = P.causal ? min(s.lk, s.lk - s.lq + min(s.lq, (w.t + 1) * P.tokens)) : s.lk;
    it.b = who[lo];
    it.h = w.h;
    it.t = w.t;
    it.q_start = s.q0;
    it.lq = s.lq;
    it.lk = s.lk;
    it.j0 = 0;
    it.j1 = kv_end > 0 ? tiles_for(kv_end, kBlockN) : 0;
    it.slot = -1;
    return it.j1;
  };
  // Every tile whole; the units of all of them, of the largest and of the smallest.
  __shared__ int most_s, least_s;
  if (tid == 0) {
    most_s = 0;
    least_s = INT_MAX;
  }
  int sum = 0, most = 0, least = INT_MAX;
  for (int x = tid; x < W; x += kPlanThreads) {
    PlanItem it;
    const int n = max(1, tile_at(x, it));
    sum += n;
    most = max(most, n);
    least = min(least, n);
    P.items[x] = it;
  }
  const int all = block_total(block_scan(sum, sums));
  atomicMax(&most_s, most);
  atomicMin(&least_s, least);
  __syncthreads();
  // When the last CTA is done, in units, a tile adding two: equal tiles go in
  // rounds, unequal ones (the longest first) end within half a small one of
  // each other.
  const int rounds = (W + P.ctas - 1) / P.ctas, share = (all + P.ctas - 1) / P.ctas;
  const int uneven = max(most_s + 2, share + least_s / 2 + 2 * rounds);
  const int uncut = 4 * least_s >= 3 * most_s ? rounds * (most_s + 2) : uneven;
  const int waves = W / P.ctas - (B > 1 ? 1 : 0), shares = P.ctas * (B > 1 ? 2 : 1);
  const int even = waves > 0 ? waves * P.ctas : 0;
  const int whole = uncut <= share + 8 + (W - even + shares) / 18 ? W : even;
  // The cut tiles: fewer than two waves (and than this block's threads).
  const int cut = W - whole;
  PlanItem it;
  int units = 0;
  if (tid < cut) units = max(1, tile_at(whole + tid, it));
  const int u1 = block_scan(units, sums), u0 = u1 - units;
  const int total = block_total(u1);
  const int size = max(kMinPieceUnits, (total + shares - 1) / shares);
  const int pieces = (total + size - 1) / size;
  if (tid < cut) {
    const int p0 = u0 / size, p1 = (u1 - 1) / size;
    PlanCut c;
    c.item = it;
    c.item.slot = p0 + tid;
    c.parts = p1 - p0 + 1;
    P.cuts[tid] = c;
    for (int p = p0; p <= p1; ++p) {
      PlanItem sgm = it;
      sgm.j0 = max(u0, p * size) - u0;
      sgm.j1 = min(it.j1, min(u1, (p + 1) * size) - u0);   // (a tile that sees no key is one unit)
      sgm.slot = p0 == p1 ? -1 : p + tid;
      P.items[whole + p + tid] = sgm;
      // the piece's first segment, and (from its last one) how many there are
      if (u0 <= p * size) P.pieces[p].first = whole + p + tid;
      if (u1 >= (p + 1) * size || tid == cut - 1) P.pieces[p].last = whole + p + tid;
    }
  }
  if (tid == 0) {
    P.head->whole = whole;
    P.head->pieces = pieces;
    P.head->cut = cut;
  }
}

// One warp per row of a cut tile: O = sum exp(L_p - L) O_p, L = log sum exp(L_p)
// over the tile's parts.
constexpr int kMergeWarps = 8;
template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32) paged_tile_merge_kernel(const __grid_constant__ PlanParams P) {
  constexpr int C = D / 32;
  ptx::grid_dependency_wait();
  if ((int)blockIdx.x >= P.head->cut) return;
  const PlanCut c = P.cuts[blockIdx.x];
  if (c.parts < 2) return;
  const int row = blockIdx.y * kMergeWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int r = row & (kBlockM - 1), in_tile = r / P.pack;   // row of its MMA tile, its token
  const int tok = c.item.t * P.tokens + (row / kBlockM) * P.pack_tokens + in_tile;
  if (in_tile >= P.pack_tokens) return;
  if (tok >= c.item.lq) return;
  const int h = c.item.h * P.pack + (r - in_tile * P.pack);
  const int64_t at = (int64_t)c.item.slot * kRowsPerTile + row;
  float mx = -INFINITY;
  for (int p = lane; p < c.parts; p += 32) mx = fmaxf(mx, P.lse_part[at + (int64_t)p * kRowsPerTile]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
  const float base = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f, acc[C];
#pragma unroll
  for (int e = 0; e < C; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int p = 0; p < c.parts; ++p) {
    const int64_t x = at + (int64_t)p * kRowsPerTile;
    const float w = expf(P.lse_part[x] - base);
    const float* v = P.o_part + x * D + C * lane;
    sum += w;
    if constexpr (C == 4) {
      const float4 t = __ldcs(reinterpret_cast<const float4*>(v));
      acc[0] = fmaf(w, t.x, acc[0]);
      acc[1] = fmaf(w, t.y, acc[1]);
      acc[2] = fmaf(w, t.z, acc[2]);
      acc[3] = fmaf(w, t.w, acc[3]);
    } else {
      const float2 t = __ldcs(reinterpret_cast<const float2*>(v));
      acc[0] = fmaf(w, t.x, acc[0]);
      acc[1] = fmaf(w, t.y, acc[1]);
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t* o = P.o + (P.s.cu_q != nullptr ? 0 : (int64_t)c.item.b * P.o_b) + (int64_t)(c.item.q_start + tok) * P.o_t +
                h * P.o_h + C * lane;
  if constexpr (C == 4)
    *reinterpret_cast<uint2*>(o) =
        make_uint2(ptx::pack_bf16(acc[0] * inv, acc[1] * inv), ptx::pack_bf16(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = ptx::pack_bf16(acc[0] * inv, acc[1] * inv);
  if (P.lse != nullptr && lane == 0) {
    const int64_t x = P.s.cu_q != nullptr ? (int64_t)h * P.s.total_q + c.item.q_start + tok
                                          : ((int64_t)c.item.b * P.heads_total + h) * P.s.seqlen_q + tok;
    P.lse[x] = sum == 0.f ? -INFINITY : mx + logf(sum);
  }
}

}  // namespace

cudaError_t paged_plan_launch(const PlanParams& p, cudaStream_t stream) {
  return launch_dependent(paged_plan_kernel, p, dim3(1), kPlanThreads, 0, stream);
}

cudaError_t paged_tile_merge_launch(const PlanParams& p, int head_dim, int max_cut, cudaStream_t stream) {
  const dim3 grid((unsigned)max_cut, kRowsPerTile / kMergeWarps);
  return head_dim == 128 ? launch_dependent(paged_tile_merge_kernel<128>, p, grid, kMergeWarps * 32, 0, stream)
                         : launch_dependent(paged_tile_merge_kernel<64>, p, grid, kMergeWarps * 32, 0, stream);
}

}  // namespace af
