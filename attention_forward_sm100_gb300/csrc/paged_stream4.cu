// Attention of a few new tokens over a paged cache of e2m1 codes.
//
// The work, its division among CTAs and the joining of parts are those of
// paged_stream.cu (paged_walk.cuh). What differs is that 4-bit keys are so few
// bytes that the instructions of loading and converting them bound the kernel, not
// HBM: 16 keys of one head of 128 depths are 2432 bytes, 103 cycles of an SM at the
// copy rate, and about 250 warp instructions at best. So
//   * a warp of its own loads: TMA boxes for the codes of up to a tile's keys of a
//     page, bulk copies for the two kinds of scales, six copies for every page of a
//     tile by four lanes (K's and V's codes; two kinds of scales each). In pages of 16
//     slots the lanes copy the scales themselves, 16 bytes at a time.
//   * four warps compute, each on 32 keys of a tile of 128 (with 32 rows two warps
//     share their keys), three CTAs per SM, two for more than 8 rows.
//   * codes become f16 two at a time and are multiplied by their block's scale,
//     which is exact (two significant bits times four). S^T = K Q^T and O^T = V^T P^T
//     as in paged_stream.cu; the vectors' scales are applied to the fp32 scores and
//     weights. For V^T, whose operands are pairs of keys, two keys' bytes are merged
//     into (key, key) pairs of a depth before they are converted.
//   * a CTA has at most two parts of segments that others have parts of too, its first
//     piece and its last. The first is counted in when it has been left, but whether it
//     is the last to come, and joins, is looked at in the end.
// Measured, GQA 32/8, 128 depths: 16 sequences of up to 32768 keys 78 us (floor 54, the
// loads alone 68), 64 of up to 8192 82 (50), one of 777 9.9; 24 of up to 4097, five new
// tokens, 16 heads of 64 depths, pages of 16 slots, 35 (11). Issue bounds it: 632 warp
// instructions for 32 keys of a head (smsp__inst_executed of the first of these, loading,
// start and end included) take 57 % of the slots in the mean and 50 % of the integer
// pipe's; a warp waits for a fixed latency 1.3 times per instruction issued, for its turn
// 0.9, for a pipe 0.7, for memory 0.7, for its next instruction 0.3.
// Tried (us for these, with 44 for the last, in this order, and a step of 32 sequences of up to 4096 with rotation
// and append, 41.5):
//   each thread copying its own 16-byte pieces (cp.async): 96, 97, 9.7, 42, -
//   one CTA of 16 warps per SM, two or three that load, two that join and store: 82, 91,
//     13, 40, 59 (with an append of 13 us in it, in place of 6)
//   the first part counted in and joined where it ends (5 us of a fence and an atomic
//     while loads are under way): 85, 89, 10.4, 45, 45.5
//   both parts counted in at the end: 79, 84, 10.3, 46, 44; by the loading warp, meanwhile:
//     78, 82, 10.4, 45.6, 41.5
//   shares of the units by the order in which an SM's CTAs start (the first has its
//     instructions issued first and ends 10 % earlier): 1 us less for the long ones, 1 to
//     2 us more for the short ones
//   the products with V in a rolled loop, for fewer instructions: 81, 83, -, -, 42
// Slots at or past the sequence's end are loaded with the rest of their page but
// their scales are set to zero, so whatever they hold cannot reach a result (codes
// are always finite).
//
// Every wait is bounded. When one runs out, the error is recorded, and with it that the
// counters of the joins may be left as they are (attn_fwd_check clears them); no wait of
// that CTA lasts any more, the computing warps leave their piece after that tile, without
// results, and end, and the loading warp ends at the next tile that is not given back,
// when its copies are there. (The way out of the loop is its count: a branch out of it,
// and the loading warp asking for each tile, cost 1.5 %.)
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "launch.cuh"
#include "paged_walk.cuh"

namespace af {
namespace {

constexpr int kThreads = 128;         // that compute
constexpr int kAll = kThreads + 32;   // and the warp that loads

template <int D_, int NT_, int WM_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WM = WM_;
  static constexpr int RT = 8 * NT * WM, WK = 4 / WM;
  static constexpr int KW = 32, NB = KW / 16;    // keys of a group per tile, 16-key blocks of them
  static constexpr int TILE = KW * WK;
  static_assert(TILE == stream4_tile(RT), "as the launch is planned");
  static constexpr int CTAS = stream4_ctas(RT);
  static constexpr int ROWB = D / 2, BK = D / 16;   // bytes of a row's codes, block scales of it
  static constexpr int VB = D / 64;                 // 4-byte words of codes that a lane holds of a key of V
  // a stage: codes of K and V, block scales of both, scales of both
  static constexpr int AT_V = TILE * ROWB, AT_KB = 2 * AT_V, AT_VB = AT_KB + TILE * BK, AT_KS = AT_VB + TILE * BK,
                       AT_VS = AT_KS + 4 * TILE, STAGE = AT_VS + 4 * TILE;
  static_assert(STAGE % 512 == 0 && AT_V % 512 == 0, "the swizzle's pattern");
  static constexpr int PART = RT * D * 4;           // a group's part of O
  static constexpr int PIECES = 4;                  // pieces that the loading warp is ahead at most
  static constexpr int QF = WM * NT * (D / 16) * 32 * 8;   // q as the instructions want it, a pair of words per lane
  static_assert(QF <= WK * PART, "where the parts go at the end of a piece");
  static constexpr int REST = WK * PART + WK * RT * 8 + 512;
  static constexpr int STAGES = min_int(8, (232448 / CTAS - 1024 - REST) / STAGE);
  static constexpr int AT_PART = STAGES * STAGE, AT_Q = AT_PART, AT_ML = AT_PART + WK * PART,
                       AT_PIECE = AT_ML + WK * RT * 8,
                       AT_BAR = AT_PIECE + (PIECES + 1) * 48, SMEM = STAGES * STAGE + REST;
  static_assert(STAGES >= 3, "loads in flight");
  static_assert((PIECES + 1) * 48 + 16 * (STAGES + PIECES) <= 512, "room for pieces and barriers");
  static constexpr int FT = kThreads;   // those that compute finish a piece
  __device__ static int ftid() { return threadIdx.x; }
  __device__ static void fsync() { ptx::bar_sync(0, kThreads); }
  __device__ static int part_col(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }
  // lane t's depths of a key: D / 4 from t D / 4 on, four for each q pair
  static constexpr int Q_STEP = 2;
  __device__ static int q_depth(int kk, int t) { return D / 4 * t + 4 * kk; }
  // Where TMA's swizzle puts 16-byte piece `c` of row `r`.
  __device__ static int swz(int r, int c) { return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1); }
  // Which row of an 8-key group is key m of the instructions (any order will do, as
  // long as K and V agree): this one spreads the rows that lanes read together, 2 t of
  // V and two (D = 64: four) neighbours of K, over all banks.
  __device__ static int key_row(int m) { return D == 128 ? m ^ ((m >> 1) & 1) : m ^ ((m >> 2) & 1); }
};

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Barriers (8 bytes each) and what is shared through them.
struct Pipe {
  uint32_t full, empty;     // of stage 0: a tile is there, its four warps are done with it
  uint32_t named, taken;    // of piece 0: a piece is described, its four warps are done with it
  int* pieces;              // 12 words each
  volatile int* over;       // a wait has run out
  uint32_t* ws;
  uint64_t limit;           // of a wait, in ns

  // False when it ran out, in this warp or before in another of the CTA.
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int role) const {
    return __all_sync(kFull, ptx::mbar_try_wait(bar, parity) || wait_long(bar, parity, role));
  }
  __device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, int role) const {
    uint64_t since = 0;
    for (uint32_t i = 1;; ++i) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if ((i & 15u) == 0u) {
        if (*over) return false;
        const uint64_t now = ptx::globaltimer();
        if (since == 0) since = now;
        if (now - since > limit) {
          atomicExch(&ws[kWsCountersLeft], 1u);
          if (atomicCAS(&ws[kWsErrorCode], 0u, (uint32_t)kDevErrTimeout) == 0u)
            atomicExch(&ws[kWsErrorInfo], (blockIdx.x << 16) | ((uint32_t)role << 8));
          *over = 1;
          return false;
        }
      }
    }
  }
};

// A piece, its sequence's rows and its first unit among all, as the loading warp
// hands them to the others; count 0: there are no more.
struct Job {
  Piece pc;
  SeqRows s;
  int first;
};
template <class C>
__device__ __forceinline__ bool hand_over(const Pipe& pipe, int k, const Job& j) {
  if (!pipe.wait(pipe.taken + 8 * (k % C::PIECES), (uint32_t)(k / C::PIECES + 1) & 1u, 2)) return false;
  if ((threadIdx.x & 31) == 0) {
    int4* to = reinterpret_cast<int4*>(pipe.pieces + 12 * (k % C::PIECES));
    to[0] = make_int4(j.pc.b, j.pc.seg, j.pc.first, j.pc.count);
    to[1] = make_int4(j.pc.tiles, j.s.lq, j.s.lk, j.s.q0);
    to[2] = make_int4(j.first, 0, 0, 0);
    ptx::mbar_arrive(pipe.named + 8 * (k % C::PIECES));
  }
  __syncwarp();
  return true;
}
__device__ __forceinline__ Job job_in(const Pipe& pipe, int place) {
  const int4* from = reinterpret_cast<const int4*>(pipe.pieces + 12 * place);
  const int4 a = from[0], b = from[1];
  return {{a.x, a.y, a.z, a.w, b.x}, {b.y, b.z, b.w}, from[2].x};
}
template <class C>
__device__ __forceinline__ Job job_at(const Pipe& pipe, int k) { return job_in(pipe, k % C::PIECES); }

// Whether scales are loaded by the lanes, 16 bytes each, and not by bulk copies, of which
// pages of few slots take very many small ones. us, by copies / by lanes: pages of 16
// slots, 24 sequences of up to 4097 keys, five new tokens, 16 heads of 64 depths 44.3 /
// 34.6; 8 heads of 128 and pages of 32, a step of 32 sequences of up to 4096, 42.6 / 43.7;
// of 64, 64 sequences of up to 8192, 81.8 / 86.1. (Kernels of their own: with both in one,
// pages of 32 slots and more lost 4 to 9 %, to the instruction cache.)
bool small_pages(const StreamParams& P) { return P.c.page_shift < 5; }

// The warp that loads: every tile of this CTA's pieces, in order. SMALL as small_pages().
template <class C, bool SMALL>
__device__ __forceinline__ void load_tiles(const Stream4Params& P, Walker<C> walk, const Pipe& pipe, uint32_t ring, int x,
                                           int end) {
  const int lane = threadIdx.x & 31;
  // A tile is units of as many keys as lie in one page. Lanes take units (of up to
  // eight, the smallest page having 16 keys) and one or two of their six copies.
  const int unit = min(C::TILE, 1 << P.c.page_shift), units = C::TILE / unit;
  const int u = lane & 7, what = lane >> 3;   // 0: codes of K, 1: of V, 2: scales of K, 3: of V
  const int page_mask = (1 << P.c.page_shift) - 1;
  const uint32_t unit_bytes = unit * (2 * C::ROWB + (SMALL ? 0 : 2 * C::BK + 8));
  int count = 0, k = 0;
  bool ok = true;
  while (ok && x < end) {
    SeqRows s;
    const Piece pc = walk.at(P, x, end, s);
    if (!(ok = hand_over<C>(pipe, k++, {pc, s, x}))) break;
    x += max(1, pc.count);
    int t0, n;
    piece_tiles<C>(P, pc, s, t0, n);
    const int hk = head_of(P, pc.seg);
    const int32_t* table = P.c.table + (int64_t)pc.b * P.c.table_stride;
    int key = t0 * C::TILE + u * unit;
    auto page_of = [&](int k) { return u < units && k < s.lk ? __ldg(table + (k >> P.c.page_shift)) : 0; };
    int page = n > 0 ? page_of(key) : 0;
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++count, key += C::TILE) {
      const bool there = u < units && key < s.lk;
      if (there) page = checked_page(P.c, page, pc.b, P.ws);
      const int next = j + 1 < n ? page_of(key + C::TILE) : 0;   // (a tile ahead)
      const int st = count % C::STAGES;
      const uint32_t bar = pipe.full + 8 * st, at = ring + st * C::STAGE;
      if (!(ok = pipe.wait(pipe.empty + 8 * st, (uint32_t)(count / C::STAGES + 1) & 1u, 1))) break;
      const unsigned have = __ballot_sync(kFull, there && what == 0);
      if (lane == 0) ptx::mbar_expect_tx(bar, __popc(have) * unit_bytes);
      __syncwarp();
      if (there) {
        const int slot = key & page_mask;
        if (what < 2)
          ptx::tma_load_4d(at + (what ? C::AT_V : 0) + u * unit * C::ROWB, what ? &P.tm_v : &P.tm_k, bar, 0, hk, slot, page);
        if (SMALL || what >= 2) {
          const int64_t first = (((int64_t)page * P.c.heads_kv + hk) << P.c.page_shift) + slot;
          if constexpr (SMALL) {
            // 16-byte pieces what, what + 4, ... of the unit's scales
            const int n4 = unit / 4, nb = unit * C::BK / 16;
            for (int c = what; c < n4; c += 4) {
              const uint32_t to = at + u * unit * 4 + c * 16;
              ptx::cp_async16(to + C::AT_KS, P.c.k_scale + first + c * 4);
              ptx::cp_async16(to + C::AT_VS, P.c.v_scale + first + c * 4);
            }
            for (int c = what; c < nb; c += 4) {
              const uint32_t to = at + u * unit * C::BK + c * 16;
              ptx::cp_async16(to + C::AT_KB, P.blocks.k + first * C::BK + c * 16);
              ptx::cp_async16(to + C::AT_VB, P.blocks.v + first * C::BK + c * 16);
            }
          } else {
            const uint8_t* blocks = what == 2 ? P.blocks.k : P.blocks.v;
            const float* scales = what == 2 ? P.c.k_scale : P.c.v_scale;
            ptx::bulk_load(at + (what == 2 ? C::AT_KB : C::AT_VB) + u * unit * C::BK, blocks + first * C::BK, unit * C::BK, bar);
            ptx::bulk_load(at + (what == 2 ? C::AT_KS : C::AT_VS) + u * unit * 4, scales + first, unit * 4, bar);
          }
        }
      }
      if constexpr (SMALL) {
        __syncwarp();
        ptx::cp_async_arrive(bar);
      }
      page = next;
    }
  }
  if (ok) hand_over<C>(pipe, k, {{0, 0, 0, 0, 1}, {0, 0, 0}, 0});
  // Nothing is left in flight when the CTA ends (but after a wait that ran out, all of
  // this has been waited for).
  for (int j = max(0, count - C::STAGES); j < count; ++j) {
    const uint64_t since = ptx::globaltimer();
    while (!ptx::mbar_try_wait(pipe.full + 8 * (j % C::STAGES), (uint32_t)(j / C::STAGES) & 1u) &&
           ptx::globaltimer() - since < pipe.limit) {
    }
  }
}

// Runs piece k. `qf` holds q of the piece, then of the
// next: its loads are on their way while this one is finished. False after the last.
template <class C>
__device__ __forceinline__ bool run_piece(const Stream4Params& P, uint8_t* smem, const Pipe& pipe, int k,
                                          uint32_t (&qf)[C::NT][C::D / 16][2], int& count, int per, bool& waits, uint32_t& early) {
  constexpr int D = C::D, WM = C::WM, NT = C::NT, KW = C::KW, NB = C::NB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3, gk = C::key_row(g);
  const int wm = warp % WM, kg = warp / WM;
  int t0, n, lk, lim_min;

  // Rows row0 + 8 x + 2 t and + 1 are this lane's columns of the score and output
  // tiles: the keys they see, and the factor of their scaled q.
  int lim[NT][2];
  {
    const Job job = job_at<C>(pipe, k);
    const int rows = job.s.lq * P.group, row0 = row_tile_of(P, job.pc.seg) * C::RT + 8 * NT * wm;
    piece_tiles<C>(P, job.pc, job.s, t0, n);
    lim_min = lk = job.s.lk;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = row0 + 8 * x + 2 * t + e;
        // (rows past the segment's end compute on zeros and are not stored)
        lim[x][e] = P.causal && r < rows ? min(lk, lk - job.s.lq + r / P.group + 1) : lk;
        lim_min = min(lim_min, lim[x][e]);
      }
  }
  lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, 1));
  lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, 2));
  float qscale[NT][2];

  const uint32_t at_q = C::AT_Q + (wm * NT * (D / 16) * 32 + lane) * 8;
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    // q as f16, times the power of two that brings its largest magnitude to
    // [2^14, 2^15): exact down to 2^-38 of that
    uint32_t top = 0u;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        top = max(top, max(qf[x][kk][e] & 0x7fffu, (qf[x][kk][e] >> 16) & 0x7fffu));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    // 2^(14 - e) in a float's exponent; e at least -112 keeps it finite, a
    // row with infinities or NaN ends as NaN whatever the factor
    const int e = max((int)(top >> 7), 15);
    const float up = __uint_as_float((uint32_t)min(268 - e, 254) << 23);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint32_t w = qf[x][kk][c];
        qf[x][kk][c] = ptx::pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
      }
    // (all key groups hold the same q and write the same words)
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
      *reinterpret_cast<uint2*>(smem + at_q + (x * (D / 16) + kk) * 256) = make_uint2(qf[x][kk][0], qf[x][kk][1]);
    const float down = __uint_as_float((uint32_t)max(e - 14, 1) << 23);
    qscale[x][0] = __shfl_sync(kFull, down, 8 * t) * P.scale_log2;
    qscale[x][1] = __shfl_sync(kFull, down, 8 * t + 4) * P.scale_log2;
  }

  ptx::bar_sync(0, kThreads);
  // O^T: depths by rows, D / 16 tiles of 16 depths
  float acc[D / 16][NT][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][x][e] = 0.f;
  // The accumulator is in units of vref / 2^7, vref a power of two at least as large
  // as every vector's scale of V so far. While the scales of a step are within 2^-4 of
  // it, weights (times scale / vref * 2^7, at most 2^15) and values (code * block
  // scale, at most 2688) are multiplied as f16: its spacing near zero, 2^-24, then
  // costs a key less than 2^-28 of the largest weight, so 2^20 keys less than bf16's
  // rounding. Steps with smaller scales go through bf16. vref is 2^-100 at least:
  // 128 / vref stays finite, and a weight times the smallest scale, 2^-126, keeps
  // bf16's bits.
  constexpr float kLeastVref = 0x1p-100f;
  float vref = 0.f, vinv = 0.f;
  // Weights are 2^(score - off), in log2 units; a row that has seen no key has set
  // false, off = 0 and l = 0.
  float off[NT][2], l[NT][2];
  bool set[NT][2], all_set = false;
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      off[x][e] = 0.f;
      l[x][e] = 0.f;
      set[x][e] = false;
    }
  // This lane's places in a stage (added to constants, the swizzle depending on the
  // row among eight alone): its key of K, the words of two keys of V, their scales.
  const int wk = kg * KW;
  const uint32_t smem0 = ptx::smem_u32(smem);
  const uint32_t at_k = (wk + gk) * C::ROWB + (D == 128 ? C::swz(gk, t) * 16 : C::swz(gk, t >> 1) * 16 + (t & 1) * 8);
  const uint32_t at_kb = C::AT_KB + (wk + gk) * C::BK + (D == 128 ? 2 * t : t);
  const uint32_t at_sc = C::AT_KS + (wk + gk) * 4;
  uint32_t at_v[2], at_vb[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = C::key_row(2 * t + e);
    at_v[e] = C::AT_V + (wk + r) * C::ROWB + (D == 128 ? C::swz(r, g >> 1) * 16 + (g & 1) * 8 : C::swz(r, g >> 2) * 16 + (g & 3) * 4);
    at_vb[e] = C::AT_VB + (wk + r) * C::BK + (D == 128 ? g : g >> 1);
  }
  int stage = count % C::STAGES, key0 = t0 * C::TILE + wk;
  uint32_t parity = (uint32_t)(count / C::STAGES) & 1u;
  count += n;

#pragma unroll 1
  for (int j = 0; j < n; ++j, key0 += C::TILE) {
    const uint32_t st = smem0 + stage * C::STAGE;
    if (!pipe.wait(pipe.full + 8 * stage, parity, 0)) n = 0;   // (this piece comes to nothing)
    if (key0 + KW > lk) {
      // slots behind the end: zero scales
      if (key0 + lane >= lk) {
        float* const ks = reinterpret_cast<float*>(smem + stage * C::STAGE + C::AT_KS) + wk + lane;
        ks[0] = ks[C::TILE] = 0.f;
        uint32_t* const kb = reinterpret_cast<uint32_t*>(smem + stage * C::STAGE + C::AT_KB + (wk + lane) * C::BK);
#pragma unroll
        for (int i = 0; i < C::BK / 4; ++i) kb[i] = kb[C::TILE * C::BK / 4 + i] = 0u;
      }
      ptx::fence_async_shared();
      __syncwarp();
    }
    // ---- S^T = K Q^T: keys g and g + 8 of each block by rows 2 t, 2 t + 1 of each column tile.
    // Lane t holds depths t D/4 .. of its keys, one or two blocks of them.
    float sc[NB][NT][4];
    uint32_t w[NB][2][D / 32];
    __half2 s2[NB][2];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][x][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * i + 8 * e;
        if constexpr (D == 128) {
          const uint4 v = ptx::ld_shared_v4(st + at_k + row * C::ROWB);
          w[i][e][0] = v.x; w[i][e][1] = v.y; w[i][e][2] = v.z; w[i][e][3] = v.w;
          s2[i][e] = as_half2(ptx::e4m3x2_to_f16x2(ptx::ld_shared_u16(st + at_kb + row * C::BK)));
        } else {
          const uint2 v = ptx::ld_shared_v2(st + at_k + row * C::ROWB);
          w[i][e][0] = v.x; w[i][e][1] = v.y;
          s2[i][e] = as_half2(ptx::e4m3x2_to_f16x2(ptx::ld_shared_u8(st + at_kb + row * C::BK)));
        }
      }
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint2 qw[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) qw[x][y] = ptx::ld_shared_v2(smem0 + at_q + (x * (D / 16) + 2 * c + y) * 256);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        uint32_t h[2][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          ptx::e2m1x8_to_f16x2(w[i][e][c], h[e]);
          const __half2 s = c < 2 ? __low2half2(s2[i][e]) : __high2half2(s2[i][e]);
#pragma unroll
          for (int y = 0; y < 4; ++y) h[e][y] = as_bits(__hmul2(as_half2(h[e][y]), s));
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const uint32_t a[4] = {h[0][2 * y], h[1][2 * y], h[0][2 * y + 1], h[1][2 * y + 1]};
#pragma unroll
          for (int x = 0; x < NT; ++x) ptx::mma_16816_f16(sc[i][x], a, qw[x][y].x, qw[x][y].y);
        }
      }
    }
    // ---- weights: 2^(score - off), the score in log2 units; where one is above 2^8, or
    // a row has no off yet, offs move to the maxima first
    float kq[NB][NT][4];   // factors of the scores
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const float k0 = ptx::ld_shared_f32(st + at_sc + 64 * i), k1 = ptx::ld_shared_f32(st + at_sc + 64 * i + 32);
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) kq[i][x][e] = qscale[x][e & 1] * (e < 2 ? k0 : k1);
    }
    auto hidden = [&](int i, int x, int e) { return key0 + 16 * i + gk + 8 * (e >> 1) >= lim[x][e & 1]; };
    float pw[NB][NT][4], most = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          pw[i][x][e] = ptx::ex2(fmaf(sc[i][x][e], kq[i][x][e], -off[x][e & 1]));
          most = fmaxf(most, pw[i][x][e]);
        }
    // (masked keys, too, are taken care of in there: the last tiles' matter alone)
    if (__any_sync(kFull, most > 256.f || key0 + KW > lim_min) || !all_set) {
      bool every = true;
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = -INFINITY;
#pragma unroll
          for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int y = e; y < 4; y += 2)
              if (!hidden(i, x, y)) v = fmaxf(v, sc[i][x][y] * kq[i][x][y]);
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 16));
          if (set[x][e] ? v > off[x][e] + 8.f : v > -INFINITY) {
            const float alpha = set[x][e] ? ptx::ex2(off[x][e] - v) : 0.f;
            off[x][e] = v;
            set[x][e] = true;
            l[x][e] *= alpha;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[i][x][e] *= alpha;
              acc[i][x][2 + e] *= alpha;
            }
          }
          every = every && set[x][e];
        }
      all_set = __all_sync(kFull, every);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            pw[i][x][e] = hidden(i, x, e) ? 0.f : ptx::ex2(fmaf(sc[i][x][e], kq[i][x][e], -off[x][e & 1]));
    }
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) l[x][e & 1] += pw[i][x][e];
    // ---- O^T += V^T P^T
    float vk[NB][2], top = 0.f, low = INFINITY;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        vk[i][e] = ptx::ld_shared_f32(st + at_sc + 4 * C::TILE + 64 * i + 32 * e);
        top = fmaxf(top, fabsf(vk[i][e]));
        low = fminf(low, fabsf(vk[i][e]));
      }
    const bool plain = __all_sync(kFull, top <= vref && low >= vref * 0.0625f);
    if (!plain) {   // a scale of 0, as behind the end, loses nothing in f16
      low = INFINITY;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) low = fminf(low, vk[i][e] == 0.f ? INFINITY : fabsf(vk[i][e]));
    }
    if (!plain && __any_sync(kFull, top > vref)) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      // the next power of two (an infinite or huge scale: 2^127; NaN leaves it)
      const uint32_t up = min(((__float_as_uint(top) + 0x7fffffu) >> 23), 254u) << 23;
      const float now = fmaxf(vref, fmaxf(__uint_as_float(up), kLeastVref));
      const float change = vref == 0.f ? 0.f : vref / now;
      vref = now;
      vinv = 128.f / now;
#pragma unroll
      for (int q = 0; q < D / 16; ++q)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[q][x][e] *= change;
    }
    auto values = [&](auto f16) {
      constexpr uint32_t LOW = 0x0f0f0f0fu;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float w0 = vk[i][0] * vinv, w1 = vk[i][1] * vinv;
        uint32_t pf[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {   // (key, rows) pairs to (row, keys) pairs
          const float a0 = pw[i][x][0] * w0, a1 = pw[i][x][1] * w0, a2 = pw[i][x][2] * w1, a3 = pw[i][x][3] * w1;
          pf[x][0] = ptx::movmatrix_trans(decltype(f16)::value ? ptx::pack_f16(a0, a1) : ptx::pack_bf16(a0, a1));
          pf[x][1] = ptx::movmatrix_trans(decltype(f16)::value ? ptx::pack_f16(a2, a3) : ptx::pack_bf16(a2, a3));
        }
        // lane (g, t): depths g * D/8 .. + D/8, of one block, of keys 2t, 2t+1, 2t+8, 2t+9
        uint32_t v[4][C::VB], b[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + 8 * (e >> 1);
          if constexpr (D == 128) {
            const uint2 x = ptx::ld_shared_v2(st + at_v[e & 1] + row * C::ROWB);
            v[e][0] = x.x; v[e][1] = x.y;
          } else {
            v[e][0] = ptx::ld_shared_u32(st + at_v[e & 1] + row * C::ROWB);
          }
          b[e] = ptx::ld_shared_u8(st + at_vb[e & 1] + row * C::BK);
        }
        const uint32_t s01 = ptx::e4m3x2_to_f16x2(b[0] + b[1] * 256u), s23 = ptx::e4m3x2_to_f16x2(b[2] + b[3] * 256u);
#pragma unroll
        for (int w = 0; w < C::VB; ++w) {
          uint32_t h[4][4];   // even depths of keys 0 and 1, odd ones, the same of keys 2 and 3
          ptx::e2m1x8_to_f16x2((v[0][w] & LOW) | ((v[1][w] << 4) & ~LOW), h[0]);
          ptx::e2m1x8_to_f16x2(((v[0][w] >> 4) & LOW) | (v[1][w] & ~LOW), h[1]);
          ptx::e2m1x8_to_f16x2((v[2][w] & LOW) | ((v[3][w] << 4) & ~LOW), h[2]);
          ptx::e2m1x8_to_f16x2(((v[2][w] >> 4) & LOW) | (v[3][w] & ~LOW), h[3]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            uint32_t a[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              a[c] = ptx::mul_f16x2(h[c][y], c < 2 ? s01 : s23);
              if constexpr (!decltype(f16)::value) a[c] = ptx::f16x2_to_bf16x2(a[c]);
            }
#pragma unroll
            for (int x = 0; x < NT; ++x) {
              if constexpr (decltype(f16)::value) ptx::mma_16816_f16(acc[4 * w + y][x], a, pf[x][0], pf[x][1]);
              else ptx::mma_16816(acc[4 * w + y][x], a, pf[x][0], pf[x][1]);
            }
          }
        }
      }
    };
    if (plain || __all_sync(kFull, low >= vref * 0.0625f)) values(std::true_type{});
    else values(std::false_type{});
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(pipe.empty + 8 * stage);
    if (++stage == C::STAGES) {
      stage = 0;
      parity ^= 1u;
    }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[x][e] += __shfl_xor_sync(kFull, l[x][e], o);

  const bool named = __all_sync(kFull, *pipe.over == 0) &&
                     pipe.wait(pipe.named + 8 * ((k + 1) % C::PIECES), (uint32_t)((k + 1) / C::PIECES) & 1u, 3);
  bool more = false;
  if (named) {
    const Job next = job_at<C>(pipe, k + 1);
    more = next.pc.count > 0;
    if (more) load_q<C>(P, next.pc, next.s, wm, qf);
  }

  // ---- The key groups' results meet in shared memory.
  // (nobody reads q any more, whose place it is; nor, once a tile or a piece has not come
  // in time, does any warp go on)
  if (ptx::bar_any(0, kThreads, !named)) return false;
  float2* ml = reinterpret_cast<float2*>(smem + C::AT_ML);   // [WK][RT]
  if (n > 0) {
    float* part = reinterpret_cast<float*>(smem + C::AT_PART + kg * C::PART);   // [RT][D]
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * (NT * wm + x) + 2 * t + e;
        float* dst = part + r * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          *reinterpret_cast<float2*>(dst + C::part_col(r, g * (D / 8) + 2 * i)) =
              make_float2(acc[i][x][e] * (vref * 0.0078125f), acc[i][x][2 + e] * (vref * 0.0078125f));
      }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (g == 0)
        ml[kg * C::RT + 8 * (NT * wm + x) + 2 * t + e] = make_float2(set[x][e] ? off[x][e] : -INFINITY, l[x][e]);
  ptx::bar_sync(0, kThreads);
  const Job job = job_at<C>(pipe, k);
  auto part_of = [&](int i) { return n > 0 ? reinterpret_cast<const float*>(smem + C::AT_PART + i * C::PART) : nullptr; };
  leave_piece<C>(P, job.pc, job.s, ml, part_of);
  const bool whole = job.pc.count == job.pc.tiles;
  if (more) {
    ptx::bar_sync(0, kThreads);   // (before the next piece's q is where the parts are)
    if (!whole && threadIdx.x == 0) {   // (k is 0)
      // counted in now, looked at in the end
      __threadfence();
      early = atomicAdd(PartOf(P, job.pc, job.first, per).counter(P), 1u);
      int4* to = reinterpret_cast<int4*>(pipe.pieces + 12 * C::PIECES);
      const int4* from = reinterpret_cast<const int4*>(pipe.pieces);
      to[0] = from[0]; to[1] = from[1]; to[2] = from[2];
    }
  }
  if (k == 0) waits = more && !whole;
  __syncwarp();
  if (lane == 0 && more) ptx::mbar_arrive(pipe.taken + 8 * (k % C::PIECES));
  if (!more) {
    // The last piece's segment, then the first one's. (More rows have their joins in one
    // place, the instructions for the second one then being in the cache: 8 sequences of up
    // to 1000 keys, 32 rows of 128 depths, 36 us instead of 44; 8 rows are done sooner
    // without the loop.)
    auto join = [&](bool last) {
      if (!last) ptx::bar_sync(0, kThreads);
      const Job j = last ? job : job_in(pipe, C::PIECES);
      join_piece<C>(P, j.pc, j.s, j.first, per, !last, early);
    };
    if constexpr (C::RT == 8) {
      if (!whole) join(true);
      if (waits) join(false);
    } else {
#pragma unroll 1
      for (int i = whole ? 1 : 0; i <= (waits ? 1 : 0); ++i) join(i == 0);
    }
  }
  return more;
}

template <int D, int NT, int WM, bool SMALL>
__global__ void __launch_bounds__(kAll, (Cfg<D, NT, WM>::CTAS))
    paged_stream4_kernel(const __grid_constant__ Stream4Params P) {
  using C = Cfg<D, NT, WM>;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int over;
  Pipe pipe;
  pipe.full = ptx::smem_u32(smem) + C::AT_BAR;
  pipe.empty = pipe.full + 8 * C::STAGES;
  pipe.named = pipe.empty + 8 * C::STAGES;
  pipe.taken = pipe.named + 8 * C::PIECES;
  pipe.pieces = reinterpret_cast<int*>(smem + C::AT_PIECE);
  pipe.over = &over;
  pipe.ws = P.ws;
  pipe.limit = P.timeout_ns;
  if (threadIdx.x == 0) {
    over = 0;
#pragma unroll
    for (int i = 0; i < C::STAGES; ++i) {
      // (the lanes' arrivals; to withhold a tile, one more, that nobody makes)
      ptx::mbar_init(pipe.full + 8 * i, (SMALL ? 33 : 1) + (i == 0 && blockIdx.x == 0 ? P.withhold : 0));
      ptx::mbar_init(pipe.empty + 8 * i, kThreads / 32);
    }
#pragma unroll
    for (int i = 0; i < C::PIECES; ++i) {
      ptx::mbar_init(pipe.named + 8 * i, 1);
      ptx::mbar_init(pipe.taken + 8 * i, kThreads / 32);
    }
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&P.tm_k);
    ptx::prefetch_tmap(&P.tm_v);
  }
  __syncthreads();
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  // Every warp needs the units of a CTA, the loading one also where to find them.
  Walker<C> walk;
  const int total = walk.start(P);
  const int teams = (int)gridDim.x / P.team;
  const int per = (total + teams - 1) / teams, team = (int)blockIdx.x / P.team;
  int x = min(total, team * per);
  const int end = min(total, x + per);
  if (x >= end) return;
  if (threadIdx.x >= kThreads) {
    if (P.s.batch > 32) walk.seek(P, x);
    load_tiles<C, SMALL>(P, walk, pipe, ptx::smem_u32(smem), x, end);
    return;
  }
  uint32_t qf[C::NT][D / 16][2];
  if (ptx::bar_any(0, kThreads, !pipe.wait(pipe.named, 0u, 3))) return;
  {
    const Job job = job_at<C>(pipe, 0);
    load_q<C>(P, job.pc, job.s, (int)(threadIdx.x >> 5) % C::WM, qf);
  }
  int count = 0;   // tiles used so far
  // a first piece that is a part, counted in as this one from 0
  bool waits = false;
  uint32_t early = 0u;
  for (int k = 0; run_piece<C>(P, smem, pipe, k, qf, count, per, waits, early); ++k) {
  }
}

template <int D, int NT, int WM, bool SMALL>
cudaError_t launch_s(const Stream4Params& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, NT, WM>;
  constexpr auto kern = paged_stream4_kernel<D, NT, WM, SMALL>;
  return launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), kAll, C::SMEM, stream); });
}

template <int D, int NT, int WM>
cudaError_t launch_t(const Stream4Params& p, int grid, cudaStream_t stream) {
  return small_pages(p) ? launch_s<D, NT, WM, true>(p, grid, stream) : launch_s<D, NT, WM, false>(p, grid, stream);
}

template <int D>
cudaError_t launch_d(const Stream4Params& p, int row_tile, int grid, cudaStream_t stream) {
  switch (row_tile) {
    case 8: return launch_t<D, 1, 1>(p, grid, stream);
    case 16: return launch_t<D, 2, 1>(p, grid, stream);
    default: return launch_t<D, 2, 2>(p, grid, stream);
  }
}

}  // namespace

cudaError_t paged_stream4_launch(const Stream4Params& p, int head_dim, int row_tile, int grid, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128>(p, row_tile, grid, stream) : launch_d<64>(p, row_tile, grid, stream);
}

}  // namespace af
