// Attention of a few new tokens over the paged cache: a streaming kernel for
// problems that HBM bounds.
//
// The new tokens of one sequence times the query heads that share one KV head
// are R = Lq * Hq / Hkv rows over the same keys. For few rows the cached K and V
// are all that matters: they have to cross HBM once, and R flops per byte leave
// the tensor cores idle. So the kernel is built around the loads:
//   * the work is the list of all key tiles (64 or 128 keys) of all (sequence,
//     KV head, row tile) segments, cut into equal contiguous parts, one per CTA
//     (two or three CTAs per SM). Neighbouring CTAs share a cut and differ in
//     the head, so that HBM is asked for what lies together (182 -> 171 us, e4m3
//     125 -> 106 at the sizes given at kMaxTeam). Lengths are read on the device,
//     so ragged batches balance without the host knowing them and a captured
//     call follows lengths that change;
//   * many short segments are bound by what is done once for each: lengths are
//     summed 256 at a time, q of the next segment is loaded while one is
//     finished, uncut segments share CTAs as cut ones do (256 sequences of up to
//     250 keys: 59 -> 39 us);
//   * a CTA streams its tiles through a ring of cp.async stages (192 KB per SM),
//     across segments: while one is finished, the next one's tiles are loading.
//     A row tile is 8, 16 or 32 rows; the four warps form four key groups, each
//     with its own keys and ring, so that every warp streams by itself and meets
//     no barrier inside a segment (with 32 rows two groups of two warps);
//   * one pass with running maximum and sum (fp32, log2 units) and m16n8k16
//     tensor instructions, keys (then depths) on the 16-wide side and rows on
//     the 8-wide one: S^T = K Q^T, O^T = V^T P^T, so up to eight rows cost half
//     the instructions, exponentials and registers of sixteen. They are too few
//     for the 128-row instructions of the tcgen05 kernel, and the loads bound
//     both. The maximum only moves when it grows by more than 2^8, so the
//     accumulator is rarely rescaled; O and the sum share it, so their quotient
//     is exact;
//   * e4m3 codes are multiplied as f16, exactly (one conversion for two of them;
//     to bf16 it takes four): q as f16 too, normalised by a power of two per row,
//     and the weights in units of the largest value scale (where scales differ
//     by more than 2^4 weights and values go through bf16). The key scale is
//     applied to the fp32 score, the value scale to the fp32 weight. Depth and
//     value columns are dealt to lanes in the order in which 16-byte reads from
//     shared memory deliver them: a dot product does not depend on the order of
//     its depth, nor a product on that of its columns;
//   * a segment that lies in one CTA is finished there; the parts of one that
//     CTA borders cut meet in the workspace, and whichever of its CTAs comes last
//     joins them (in the order of the CTAs, so the result does not depend on who
//     it is). A second kernel for that cost 4 to 7 us per call.
// Slots at or past the sequence's end are not read (their shared memory is
// zeroed), so whatever they hold cannot reach a result.
#include <math.h>

#include <type_traits>

#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace af {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int min_int(int a, int b) { return a < b ? a : b; }

// NT * 8 rows per warp, WM warps to a key group.
template <int D_, int KIND_, int NT_, int WM_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WM = WM_, KIND = KIND_;
  static constexpr bool FP8 = KIND == kE4m3, FP4 = KIND == kE2m1;
  static constexpr bool CODES = FP8 || FP4;      // codes with scales, multiplied as f16
  static constexpr int ROWB = FP4 ? D / 2 : (FP8 ? D : 2 * D);   // bytes of a cached row
  static constexpr int CTAS = stream_ctas(ROWB, 8 * NT * WM);
  static constexpr int WK = 4 / WM;              // key groups
  static constexpr int RT = 8 * NT * WM;         // rows of a row tile
  static constexpr int KW = stream_tile(ROWB, WM) / WK;   // keys of a group per tile
  static constexpr int TILE = KW * WK;
  static constexpr int BLOCKS = KW / 16;         // 16-key blocks of a group's tile
  static constexpr int CPR = ROWB / 16;          // 16-byte pieces of a row
  static constexpr int GT = 32 * WM;             // threads of a group
  static constexpr int LT = min_int(GT, 16 * CPR);   // of them, those that load rows
  static constexpr int RS = LT / CPR;            // rows a group loads at a time
  static_assert(RS <= 16, "the rows of a load lie in one 16-key block");
  static constexpr int NL = KW / RS;             // loads per thread of K (and of V)
  static constexpr int KV = KW * ROWB;
  static constexpr int SC = CODES ? KW * 4 : 0;      // a scale for every key
  static constexpr int BK = D / 16;                  // block scales of a key
  static constexpr int BL = FP4 ? KW * BK : 0;
  static constexpr int STAGE = 2 * (KV + SC + BL);   // bytes of one group's stage
  // At the end of a segment a group leaves its part of O in the stage that it
  // has just used up, or, where that is too small, in room of its own.
  static constexpr int PART = RT * D * 4;
  static constexpr bool OWN_PART = PART > STAGE;
  static constexpr int STAGES = FP4 ? min_int(8, (225280 / CTAS - (OWN_PART ? WK * PART : 0)) / (WK * STAGE))
                                    : min_int(8, (196608 / CTAS - (OWN_PART ? WK * PART : 0)) / (WK * 2 * KV));
  static constexpr int RING = WK * STAGES * STAGE;
  static constexpr int OFF_ML = RING + (OWN_PART ? WK * PART : 0);   // [WK][RT] (maximum, sum)
  static constexpr int SMEM = OFF_ML + WK * RT * 8;
  static constexpr int ROUNDS = (RT * (D / 4) + 127) / 128;   // 16-byte pieces of a row tile per thread
  // Byte offset of group k's part, `last` being its stage's in the group's ring.
  __device__ static int part_at(int k, int last) { return OWN_PART ? RING + k * PART : k * (STAGES * STAGE) + last; }
  static_assert(STAGES >= 3 && SMEM <= 226 * 1024 / CTAS, "the CTAs per SM");
  // Column of depth d of row r there: rows 2 t and 2 t + 1 shifted by 8 t banks.
  __device__ static int part_col(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }
  // Position of 16-byte piece `c` of row `r` in a stage (bank conflicts).
  __device__ static int swz_k(int r, int c) {
    if (FP4) return CPR == 4 ? c ^ ((r >> 1) & 2) : c;
    return FP8 ? (CPR == 8 ? c ^ ((r & 1) << 2) : c) : c ^ (r & 7);
  }
  __device__ static int swz_v(int r, int c) {
    if (FP4) return swz_k(r, c);
    return FP8 && CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7);
  }
  // Which row of an 8-key group is key m of the instructions (any order will do, as
  // long as K and V agree): e2m1 rows are so short that the four rows 2 t that the
  // lanes of a product with V read would lie in the same banks.
  __device__ static int key_row(int m) { return !FP4 ? m : (CPR == 4 ? m ^ ((m >> 1) & 1) : m ^ ((m >> 2) & 1)); }
};

// The CTAs work in teams of P.team neighbours, and the cut of the work is one for
// all members of a team: member i takes KV heads i, i + team, ... (head_of), so
// the members read the same keys' rows, adjacent in memory, at about the same time.
__device__ __forceinline__ int head_of(const StreamParams& P, int seg) {
  return seg % P.team_heads * P.team + (int)blockIdx.x % P.team;
}
__device__ __forceinline__ int row_tile_of(const StreamParams& P, int seg) { return seg / P.team_heads; }
// CTA of this member in team `c`.
__device__ __forceinline__ int cta_of(const StreamParams& P, int c) { return c * P.team + (int)blockIdx.x % P.team; }

// A member's work units of sequence b: row tiles * its KV heads * (key tiles, or 1
// unsplit).
struct SeqUnits {
  SeqRows r;
  int row_tiles, tiles, units;
};

template <class C>
__device__ __forceinline__ SeqUnits seq_units(const StreamParams& P, const SeqRaw& raw, int b) {
  SeqUnits u;
  u.r = checked_seq(P.s, raw, b, P.ws);
  u.row_tiles = (int)(((int64_t)u.r.lq * P.group + C::RT - 1) / C::RT);
  u.tiles = P.split ? max(1, (u.r.lk + C::TILE - 1) / C::TILE) : 1;
  u.units = u.row_tiles * P.team_heads * u.tiles;
  return u;
}

// One contiguous part of a segment.
struct Piece {
  int b, seg;            // seg = row tile * team_heads + the member's how-manieth KV head
  int first, count;      // unit range within the segment
  int tiles;             // units of the segment
};

// Inclusive sums over the lanes.
__device__ __forceinline__ int scan(int v) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFull, v, o);
    if ((int)(threadIdx.x & 31) >= o) v += n;
  }
  return v;
}

// Finds pieces in order. Lane i holds sequence b + i of the current window of 32
// and the sums of up to 32 windows, so that a CTA's first sequence, and the next
// window, are one load away (one window after another, a CTA at the end of 256
// sequences spent 4 us to get there).
template <class C>
struct Walker {
  SeqUnits u;
  int incl;              // units of the window's sequences up to and including this lane's
  int b, base;           // first sequence of the window, units in front of it
  int span, span_base;   // first sequence of these windows (1024 sequences), units in front of it
  int wincl;             // units of their windows up to and including this lane's

  // Sums of the windows from sequence `first` on, the lengths of AHEAD windows
  // being loaded at once; returns their units.
  template <int AHEAD>
  __device__ __forceinline__ int windows(const StreamParams& P, int first) {
    const int lane = threadIdx.x & 31;
    int mine = 0;
    span = first;
#pragma unroll 1
    for (int w0 = 0; w0 < 32 && first + 32 * w0 < P.s.batch; w0 += AHEAD) {
      SeqRaw raw[AHEAD];
#pragma unroll
      for (int y = 0; y < AHEAD; ++y) {
        const int c = first + 32 * (w0 + y) + lane;
        raw[y] = {0, 0, 0};
        if (c < P.s.batch) raw[y] = load_seq_raw(P.s, c);
      }
#pragma unroll
      for (int y = 0; y < AHEAD; ++y) {
        const int c = first + 32 * (w0 + y) + lane;
        const int n = __reduce_add_sync(kFull, c < P.s.batch ? seq_units<C>(P, raw[y], c).units : 0);
        if (lane == w0 + y) mine = n;
      }
    }
    wincl = scan(mine);
    return __shfl_sync(kFull, wincl, 31);
  }
  // To the window of sequence `first`, `before` units in front of it.
  __device__ __forceinline__ void window(const StreamParams& P, int first, int before) {
    const int c = first + (threadIdx.x & 31);
    b = first;
    base = before;
    u.r = {0, 0, 0};
    u.tiles = 1;
    u.units = 0;
    if (c < P.s.batch) u = seq_units<C>(P, load_seq_raw(P.s, c), c);
    incl = scan(u.units);
  }
  // To the beginning; returns the units of all sequences.
  __device__ __forceinline__ int start(const StreamParams& P) {
    if (P.s.batch <= 32) {   // (one window)
      window(P, 0, 0);
      span = span_base = 0;
      wincl = __shfl_sync(kFull, incl, 31);
      return wincl;
    }
    int n = 0;
#pragma unroll 1
    for (int c = 1024; c < P.s.batch; c += 1024) n += windows<8>(P, c);
    n += windows<8>(P, 0);
    span_base = 0;
    return n;
  }
  // To the window that holds unit x, which is not in front of these windows (at
  // the end of all units: to the last window).
  __device__ __forceinline__ void seek(const StreamParams& P, int x) {
    unsigned hit = __ballot_sync(kFull, x < span_base + wincl);
    while (hit == 0u && span + 1024 < P.s.batch) {
      span_base += __shfl_sync(kFull, wincl, 31);
      windows<1>(P, span + 1024);   // (1: this code is part of the loops)
      hit = __ballot_sync(kFull, x < span_base + wincl);
    }
    const int w = hit ? __ffs(hit) - 1 : 31;
    const int before = __shfl_sync(kFull, wincl, max(w - 1, 0));
    window(P, span + 32 * w, span_base + (w ? before : 0));
  }
  // Piece that holds unit x, cut at `end`. All lanes of the warp; x increases
  // and is in front of the last unit.
  __device__ __forceinline__ Piece at(const StreamParams& P, int x, int end, SeqRows& rows) {
    unsigned hit = __ballot_sync(kFull, x < base + incl);
    if (hit == 0u) {
      seek(P, x);
      hit = __ballot_sync(kFull, x < base + incl);
    }
    const int w = hit ? __ffs(hit) - 1 : 0;
    const int local = x - base - __shfl_sync(kFull, incl - u.units, w);
    Piece p;
    p.b = b + w;
    p.tiles = __shfl_sync(kFull, u.tiles, w);
    rows.lq = __shfl_sync(kFull, u.r.lq, w);
    rows.lk = __shfl_sync(kFull, u.r.lk, w);
    rows.q0 = __shfl_sync(kFull, u.r.q0, w);
    p.seg = local / p.tiles;
    p.first = local - p.seg * p.tiles;
    p.count = min(p.tiles - p.first, end - x);
    return p;
  }
};

// Element offsets of row `r` (token-major, the group's heads fastest) of a segment.
struct RowAt {
  int i, h;
};
__device__ __forceinline__ RowAt row_at(const StreamParams& P, int hk, int r) {
  RowAt a;
  a.i = r / P.group;
  a.h = hk * P.group + (r - a.i * P.group);
  return a;
}
__device__ __forceinline__ const uint8_t* q_row(const StreamParams& P, const SeqRows& s, int b, const RowAt& a) {
  return P.q + (P.s.cu_q != nullptr ? 0 : b * P.q_b) + (int64_t)(s.q0 + a.i) * P.q_t + a.h * P.q_h;
}
__device__ __forceinline__ int64_t lse_at(const StreamParams& P, const SeqRows& s, int b, const RowAt& a) {
  return P.s.cu_q != nullptr ? (int64_t)a.h * P.s.total_q + s.q0 + a.i
                             : ((int64_t)b * P.heads_q + a.h) * P.s.seqlen_q + a.i;
}
__device__ __forceinline__ uint16_t* o_at(const StreamParams& P, const SeqRows& s, int b, const RowAt& a) {
  return P.o + (P.s.cu_q != nullptr ? 0 : b * P.o_b) + (int64_t)(s.q0 + a.i) * P.o_t + a.h * P.o_h;
}
// Natural-log sum of exponentials from a maximum in log2 units and a sum.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : fmaf(m, 0.69314718055994531f, logf(l));
}

// Tiles [first, first + count) of key tiles of a piece (none for an empty sequence).
template <class C>
__device__ __forceinline__ void piece_tiles(const StreamParams& P, const Piece& pc, const SeqRows& s, int& t0, int& n) {
  const int key_tiles = (s.lk + C::TILE - 1) / C::TILE;
  t0 = P.split ? pc.first : 0;
  n = P.split ? min(pc.count, key_tiles - t0) : key_tiles;
}

// The loads of this CTA's tiles, in order and without regard to pieces: while
// one piece is finished the next one's tiles are already on their way. One
// loader per key group; its threads agree on everything but their part of a tile.
template <class C>
struct Loader {
  Walker<C> walk;
  int x, end;              // units not yet looked at
  int b, hk, lk;           // the current tile's sequence, KV head, keys
  int key0, left;          // its first key of this group; tiles left in the piece, this one included (0: none left)
  int pages[C::BLOCKS];    // of its 16-key blocks, as read from the table
  const uint8_t *ks, *vs;  // the KV head's keys and values, at this thread's row and depth of a block
  const int32_t* table;    // the sequence's row

  __device__ __forceinline__ void fetch_pages(const StreamParams& P) {
#pragma unroll
    for (int u = 0; u < C::BLOCKS; ++u)
      pages[u] = key0 + 16 * u < lk ? ptx::ld_global_pinned(table + ((key0 + 16 * u) >> P.c.page_shift)) : 0;
  }
  // Moves to the first tile of the next piece that has any.
  __device__ __forceinline__ void next_piece(const StreamParams& P, int gt, int kg) {
    left = 0;
    while (left <= 0 && x < end) {
      SeqRows s;
      const Piece pc = walk.at(P, x, end, s);
      x += max(1, pc.count);
      int t0;
      piece_tiles<C>(P, pc, s, t0, left);
      b = pc.b;
      hk = head_of(P, pc.seg);
      lk = s.lk;
      key0 = t0 * C::TILE + kg * C::KW;
    }
    if (left <= 0) return;
    const int lrow = gt / C::CPR, lcol = gt % C::CPR;
    ks = P.c.k + hk * P.c.k_head + lrow * P.c.k_tok + lcol * 16;
    vs = P.c.v + hk * P.c.v_head + lrow * P.c.v_tok + lcol * 16;
    table = P.c.table + (int64_t)b * P.c.table_stride;
    fetch_pages(P);
  }
  // Copies the current tile into the stage at `st` and moves on: the table is
  // read a tile ahead of the copies that depend on it.
  __device__ __forceinline__ void issue(const StreamParams& P, uint32_t st, int gt, int kg) {
    if (left <= 0) return;
    const int lrow = gt / C::CPR, lcol = gt % C::CPR;
    const int page_mask = (1 << P.c.page_shift) - 1;
#pragma unroll
    for (int u = 0; u < C::BLOCKS; ++u) pages[u] = checked_page(P.c, pages[u], b, P.ws);
    constexpr int PER = 16 / C::RS;   // loads of a 16-key block per thread
#pragma unroll
    for (int i = 0; i < C::NL; i += PER) {
      if (C::LT < C::GT && gt >= C::LT) break;
      const int page = pages[i / PER];
      const int64_t slot = (key0 + 16 * (i / PER)) & page_mask;
      const uint8_t* kp = ks + page * P.c.k_page + slot * P.c.k_tok;
      const uint8_t* vp = vs + page * P.c.v_page + slot * P.c.v_tok;
#pragma unroll
      for (int y = 0; y < PER; ++y) {
        const int row = lrow + (i + y) * C::RS;
        // (behind the end nothing is read; the address is still inside a page)
        const bool ok = key0 + row < lk;
        ptx::cp_async16(st + row * C::ROWB + C::swz_k(row, lcol) * 16, kp, ok);
        ptx::cp_async16(st + C::KV + row * C::ROWB + C::swz_v(row, lcol) * 16, vp, ok);
        kp += C::RS * P.c.k_tok;
        vp += C::RS * P.c.v_tok;
      }
    }
    if constexpr (C::FP4) {
      // block scales: 16 / BK keys per 16 bytes, cut at the end as the others
      constexpr int KP = 16 / C::BK, NP = C::KW / KP;
      static_assert(2 * NP <= C::GT, "one piece per thread");
      if (gt < 2 * NP) {
        const int which = gt / NP, k = KP * (gt % NP);
        int page = pages[0];
#pragma unroll
        for (int u = 1; u < C::BLOCKS; ++u)
          if ((k >> 4) == u) page = pages[u];
        const int bytes = min(16, max(0, lk - (key0 + k)) * C::BK);
        const uint8_t* base = which ? P.blocks.v : P.blocks.k;
        const uint8_t* src =
            bytes ? base + ((((int64_t)page * P.c.heads_kv + hk) << P.c.page_shift) + ((key0 + k) & page_mask)) * C::BK
                  : base;
        ptx::cp_async16_part(st + 2 * (C::KV + C::SC) + which * C::BL + k * C::BK, src, bytes);
      }
    }
    if constexpr (C::CODES) {
      // scales: 4 keys per 16 bytes; a piece that crosses the end is cut there
      if (gt < 2 * C::KW / 4) {
        const int which = gt / (C::KW / 4), k4 = 4 * (gt % (C::KW / 4));
        int page = pages[0];
#pragma unroll
        for (int u = 1; u < C::BLOCKS; ++u)
          if ((k4 >> 4) == u) page = pages[u];
        const int keys = lk - (key0 + k4);
        const int bytes = keys >= 4 ? 16 : (keys > 0 ? 4 * keys : 0);
        const float* base = which ? P.c.v_scale : P.c.k_scale;
        const float* src =
            bytes ? base + ((((int64_t)page * P.c.heads_kv + hk) << P.c.page_shift) + ((key0 + k4) & page_mask)) : base;
        ptx::cp_async16_part(st + 2 * C::KV + which * C::SC + k4 * 4, src, bytes);
      }
    }
    key0 += C::TILE;
    if (--left > 0) fetch_pages(P);
    else next_piece(P, gt, kg);
  }
};

// Joining the parts of a segment that several CTAs hold, the same member of
// teams c0 .. last. Each
// leaves its part (accumulator, maximum, sum) in the workspace and counts
// itself in; the last of every kJoin neighbours joins theirs into the first
// one's, the last of those neighbourhoods joins what is left and finishes the
// rows. Nobody waits, and the parts are summed in the order of their CTAs
// whoever sums them. Slot 2 c + 1 is the part of the segment that starts in CTA
// c and goes on, slot 2 c that of the one that comes from an earlier team.
constexpr int kJoin = 16;

// Whether this CTA is the last of `want` to count itself in (and leaves the
// counter at zero).
__device__ __forceinline__ bool count_in(uint32_t* counter, uint32_t want) {
  __shared__ bool is_last;
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();   // (of the whole CTA's stores: the barrier above orders them before it)
    is_last = atomicAdd(counter, 1u) == want - 1u;
    if (is_last) *counter = 0u;
    __threadfence();
  }
  __syncthreads();
  return is_last;
}

// Sums parts 0 .. n - 1 at slots slot(i) of the segment's `valid` rows; hands
// (round, row, depth, four sums, maximum, sum) to `put`, whose thread alone
// holds them (round: of this thread's, a constant after unrolling). Sixteen
// loads of a thread are in flight: up to four rows, times parts.
template <class C, class Slot, class Put>
__device__ __forceinline__ void join_parts(const StreamParams& P, int n, int valid, Slot slot, Put put) {
  constexpr int D = C::D, ROUNDS = C::ROUNDS, IT = min_int(ROUNDS, 4), PB = 16 / IT;
#pragma unroll
  for (int g = 0; g < ROUNDS / IT; ++g) {
    float mm[IT], ll[IT];
    float4 o[IT];
#pragma unroll
    for (int y = 0; y < IT; ++y) {
      mm[y] = -INFINITY;
      ll[y] = 0.f;
      o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int x0 = threadIdx.x + g * IT * kThreads;
    if (x0 >= valid * (D / 4)) break;
    for (int i0 = 0; i0 < n; i0 += PB) {
      float4 v[IT][PB];
      float2 ml[IT][PB];
#pragma unroll
      for (int i = 0; i < PB; ++i)
#pragma unroll
        for (int y = 0; y < IT; ++y) {
          const int x = x0 + y * kThreads;
          ml[y][i] = make_float2(-INFINITY, 0.f);
          v[y][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + i < n && x < valid * (D / 4)) {
            const int64_t at = slot(i0 + i) * C::RT + x / (D / 4);
            ml[y][i] = __ldcg(P.part_ml + at);
            v[y][i] = __ldcg(reinterpret_cast<const float4*>(P.part_o + at * D + 4 * (x % (D / 4))));
          }
        }
#pragma unroll
      for (int y = 0; y < IT; ++y) {
        float top = mm[y];
#pragma unroll
        for (int i = 0; i < PB; ++i) top = fmaxf(top, ml[y][i].x);
        const float base = top == -INFINITY ? 0.f : top, w = ptx::ex2(mm[y] - base);
        mm[y] = top;
        ll[y] *= w;
        o[y].x *= w; o[y].y *= w; o[y].z *= w; o[y].w *= w;
#pragma unroll
        for (int i = 0; i < PB; ++i) {
          const float wi = ptx::ex2(ml[y][i].x - base);
          ll[y] = fmaf(wi, ml[y][i].y, ll[y]);
          o[y].x = fmaf(wi, v[y][i].x, o[y].x);
          o[y].y = fmaf(wi, v[y][i].y, o[y].y);
          o[y].z = fmaf(wi, v[y][i].z, o[y].z);
          o[y].w = fmaf(wi, v[y][i].w, o[y].w);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < IT; ++y) {
      const int x = x0 + y * kThreads;
      if (x < valid * (D / 4)) put(g * IT + y, x / (D / 4), 4 * (x % (D / 4)), o[y], mm[y], ll[y]);
    }
  }
}

// q of a piece's rows: row g of each of the warp's column tiles, pairs at depths d
// and d + step of every 16. The loads stay where they are written.
template <class C>
__device__ __forceinline__ void load_q(const StreamParams& P, const Piece& pc, const SeqRows& s,
                                       uint32_t (&qf)[C::NT][C::D / 16][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = row_tile_of(P, pc.seg) * C::RT + 8 * C::NT * ((int)(threadIdx.x >> 5) % C::WM);
#pragma unroll
  for (int x = 0; x < C::NT; ++x) {
    const int r = row0 + 8 * x + g;
    const bool ok = r < s.lq * P.group;
    const uint8_t* src = q_row(P, s, pc.b, row_at(P, head_of(P, pc.seg), ok ? r : 0));
#pragma unroll
    for (int kk = 0; kk < C::D / 16; ++kk) {
      const int d = C::FP4 ? C::D / 4 * t + 4 * kk
                           : (C::FP8 ? 16 * (t + 4 * (kk >> 2)) + 4 * (kk & 3) : 16 * kk + 2 * t);
      const int step = C::CODES ? 2 : 8;
      qf[x][kk][0] = ok ? (uint32_t)ptx::ld_global_pinned(reinterpret_cast<const int*>(src + 2 * d)) : 0u;
      qf[x][kk][1] = ok ? (uint32_t)ptx::ld_global_pinned(reinterpret_cast<const int*>(src + 2 * (d + step))) : 0u;
    }
  }
}

// Runs piece `pc`, which starts at unit `first`, of a CTA whose units end at `end`,
// and finds the next one; `per`: the units of every CTA. `qf` holds q of the piece,
// then of the next: its loads are on their way while this one is finished.
template <class C>
__device__ void run_piece(const StreamParams& P, const Piece& pc, const SeqRows& s, uint8_t* smem, Loader<C>& load,
                          Walker<C>& walk, uint32_t (&qf)[C::NT][C::D / 16][2], Piece& next, SeqRows& next_rows,
                          int& count, int first, int end, int per) {
  constexpr int D = C::D, WM = C::WM, NT = C::NT, KW = C::KW, NB = C::BLOCKS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int gk = C::key_row(g);                   // row of this lane's key among eight
  const int wm = warp % WM, kg = warp / WM;
  const int gt = wm * 32 + lane;                  // thread within its key group
  const int hk = head_of(P, pc.seg), rt = row_tile_of(P, pc.seg);
  const int rows = s.lq * P.group;
  const uint32_t ring = ptx::smem_u32(smem) + kg * (C::STAGES * C::STAGE);
  int t0, n;
  piece_tiles<C>(P, pc, s, t0, n);
  const int row0 = rt * C::RT + 8 * NT * wm;      // this warp's first row

  // Rows r0 + 8 x + 2 t and + 1 are this lane's columns of the score and output
  // tiles: the keys they see, and (e4m3) the factor of their scaled q.
  int lim[NT][2], lim_min = s.lk;
  float qscale[NT][2];
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + 8 * x + 2 * t + e;
      // (rows past the segment's end compute on zeros and are not stored)
      lim[x][e] = P.causal && r < rows ? min(s.lk, s.lk - s.lq + r / P.group + 1) : s.lk;
      lim_min = min(lim_min, lim[x][e]);
    }
  lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, 1));
  lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, 2));
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    if constexpr (C::CODES) {
      // The codes of an e4m3 or e2m1 cache are multiplied as f16 (one conversion for two
      // of them). q becomes f16 too, times the power of two that brings its
      // largest magnitude to [2^14, 2^15): exact down to 2^-38 of that.
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
      const float down = __uint_as_float((uint32_t)max(e - 14, 1) << 23);
      qscale[x][0] = __shfl_sync(kFull, down, 8 * t) * P.scale_log2;
      qscale[x][1] = __shfl_sync(kFull, down, 8 * t + 4) * P.scale_log2;
    } else {
      qscale[x][0] = qscale[x][1] = P.scale_log2;
    }
  }

  auto group_sync = [&]() {
    if constexpr (WM == 1) __syncwarp();
    else ptx::bar_sync(1 + kg, C::GT);
  };

  // O^T: depths by rows, D / 16 tiles of 16 depths
  float acc[D / 16][NT][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][x][e] = 0.f;
  // Codes: the accumulator is in units of vref / 2^7, vref a power of two at
  // least as large as every value scale so far. While the scales of a step are
  // within 2^-4 of it, weights (times scale / vref * 2^7, at most 2^15) and codes
  // are multiplied as f16: its spacing near zero, 2^-24, then costs a key less
  // than 2^-28 of the largest weight, so 2^20 keys less than bf16's rounding.
  // Steps with smaller scales go through bf16. vref is 2^-100 at least: 128 / vref
  // stays finite, and a weight times the smallest scale, 2^-126, keeps bf16's bits.
  constexpr float kLeastVref = 0x1p-100f;
  float vref = 0.f, vinv = 0.f;
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[x][e] = -INFINITY;
      l[x][e] = 0.f;
    }

#pragma unroll 1
  for (int j = 0; j < n; ++j, ++count) {
    ptx::cp_async_wait<C::STAGES - 2>();
    group_sync();   // this tile has arrived, and nobody reads the previous one's stage any more
    load.issue(P, ring + ((count + C::STAGES - 1) % C::STAGES) * C::STAGE, gt, kg);
    ptx::cp_async_commit();

    const uint32_t st = ring + (count % C::STAGES) * C::STAGE;
    const int key0 = (t0 + j) * C::TILE + kg * KW;
    // ---- S^T = K Q^T: keys g and g + 8 of each block by rows 2 t, 2 t + 1 of each column tile
    float sc[NB][NT][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][x][e] = 0.f;
    if constexpr (!C::CODES) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          uint32_t a[4];
          const int row = 16 * i + (lane & 15);
          ptx::ldmatrix_x4(st + row * C::ROWB + C::swz_k(row, 2 * kk + (lane >> 4)) * 16, a);
#pragma unroll
          for (int x = 0; x < NT; ++x) ptx::mma_16816(sc[i][x], a, qf[x][kk][0], qf[x][kk][1]);
        }
    } else if constexpr (C::FP4) {
      // lane t holds depths t D/4 .. of its two keys, one or two blocks of them; codes
      // times block scales are exact in f16
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        uint32_t w[2][D / 32], s2[2][D / 64];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = 16 * i + gk + 8 * e;
          const uint32_t bl = st + 2 * (C::KV + C::SC) + row * C::BK;
          if constexpr (D == 128) {
            const uint4 v = ptx::ld_shared_v4(st + row * C::ROWB + C::swz_k(row, t) * 16);
            w[e][0] = v.x; w[e][1] = v.y; w[e][2] = v.z; w[e][3] = v.w;
            const uint32_t b = ptx::e4m3x2_to_f16x2(ptx::ld_shared_u16(bl + 2 * t));
            s2[e][0] = __byte_perm(b, b, 0x1010);
            s2[e][1] = __byte_perm(b, b, 0x3232);
          } else {
            const uint2 v = ptx::ld_shared_v2(st + row * C::ROWB + 8 * t);
            w[e][0] = v.x; w[e][1] = v.y;
            s2[e][0] = ptx::e4m3x2_to_f16x2(ptx::ld_shared_u8(bl + t) * 0x101u);
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t h[2][4];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            ptx::e2m1x8_to_f16x2(w[e][c], h[e]);
#pragma unroll
            for (int y = 0; y < 4; ++y) h[e][y] = ptx::mul_f16x2(h[e][y], s2[e][c / 2]);
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t a[4] = {h[0][2 * y], h[1][2 * y], h[0][2 * y + 1], h[1][2 * y + 1]};
#pragma unroll
            for (int x = 0; x < NT; ++x) ptx::mma_16816_f16(sc[i][x], a, qf[x][2 * c + y][0], qf[x][2 * c + y][1]);
          }
        }
      }
    } else {
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const int row = 16 * i + g;
          const uint4 w0 = ptx::ld_shared_v4(st + row * C::ROWB + C::swz_k(row, t + 4 * c) * 16);
          const uint4 w1 = ptx::ld_shared_v4(st + (row + 8) * C::ROWB + C::swz_k(row + 8, t + 4 * c) * 16);
          const uint32_t u0[4] = {w0.x, w0.y, w0.z, w0.w}, u1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t a[4];
            ptx::e4m3x4_to_f16x2(u0[e], a[0], a[2]);
            ptx::e4m3x4_to_f16x2(u1[e], a[1], a[3]);
#pragma unroll
            for (int x = 0; x < NT; ++x) ptx::mma_16816_f16(sc[i][x], a, qf[x][4 * c + e][0], qf[x][4 * c + e][1]);
          }
        }
    }
    // ---- scores in log2 units; mask; running maximum
    const float* scale_sm = reinterpret_cast<const float*>(smem + (st - ptx::smem_u32(smem)) + 2 * C::KV);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      float k0 = 1.f, k1 = 1.f;
      if constexpr (C::CODES) {
        k0 = scale_sm[16 * i + gk];
        k1 = scale_sm[16 * i + gk + 8];
      }
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[i][x][e] *= C::CODES ? qscale[x][e & 1] * (e < 2 ? k0 : k1) : qscale[x][e & 1];
    }
    if (key0 + KW > lim_min) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 16 * i + gk + 8 * (e >> 1) >= lim[x][e & 1]) sc[i][x][e] = -INFINITY;
    }
    float mx[NT][2];
    bool grow = false;
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = fmaxf(sc[0][x][e], sc[0][x][2 + e]);
#pragma unroll
        for (int i = 1; i < NB; ++i) v = fmaxf(v, fmaxf(sc[i][x][e], sc[i][x][2 + e]));
        grow = grow || v > m[x][e] + 8.f;
        mx[x][e] = v;
      }
    if (__any_sync(kFull, grow)) {   // some row's maximum may have to move (the lanes hold parts of it)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = mx[x][e];
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 4));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 8));
          v = fmaxf(v, __shfl_xor_sync(kFull, v, 16));
          if (v > m[x][e] + 8.f) {
            const float alpha = ptx::ex2(m[x][e] - v);   // 0 at the first visible key
            m[x][e] = v;
            l[x][e] *= alpha;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              acc[i][x][e] *= alpha;
              acc[i][x][2 + e] *= alpha;
            }
          }
        }
    }
    // ---- weights (a row that has seen no key yet keeps m = -inf and weights 0)
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float off = m[x][e & 1] == -INFINITY ? 0.f : m[x][e & 1];
          sc[i][x][e] = ptx::ex2(sc[i][x][e] - off);
          l[x][e & 1] += sc[i][x][e];
        }
    // ---- O^T += V^T P^T
    if constexpr (!C::CODES) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        uint32_t pf[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {   // (key, rows) pairs to (row, keys) pairs
          pf[x][0] = ptx::movmatrix_trans(ptx::pack_bf16(sc[i][x][0], sc[i][x][1]));
          pf[x][1] = ptx::movmatrix_trans(ptx::pack_bf16(sc[i][x][2], sc[i][x][3]));
        }
#pragma unroll
        for (int q = 0; q < D / 16; ++q) {
          uint32_t a[4];
          const int row = 16 * i + (lane & 7) + 8 * (lane >> 4);
          ptx::ldmatrix_x4_trans(st + C::KV + row * C::ROWB + C::swz_v(row, 2 * q + ((lane >> 3) & 1)) * 16, a);
#pragma unroll
          for (int x = 0; x < NT; ++x) ptx::mma_16816(acc[q][x], a, pf[x][0], pf[x][1]);
        }
      }
    } else {
      float vs[NB][2], top = 0.f, low = INFINITY;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          vs[i][e] = scale_sm[KW + 16 * i + gk + 8 * e];
          top = fmaxf(top, fabsf(vs[i][e]));
          // (keys behind the end have scale 0 and weight 0)
          if (key0 + 16 * i + gk + 8 * e < s.lk) low = fminf(low, fabsf(vs[i][e]));
        }
      if (__any_sync(kFull, top > vref)) {
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
      const bool as_f16 = __all_sync(kFull, low >= vref * 0.0625f);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const float w0 = vs[i][0] * vinv, w1 = vs[i][1] * vinv;
        uint32_t pf[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
          const float a0 = sc[i][x][0] * w0, a1 = sc[i][x][1] * w0, a2 = sc[i][x][2] * w1, a3 = sc[i][x][3] * w1;
          pf[x][0] = ptx::movmatrix_trans(as_f16 ? ptx::pack_f16(a0, a1) : ptx::pack_bf16(a0, a1));
          pf[x][1] = ptx::movmatrix_trans(as_f16 ? ptx::pack_f16(a2, a3) : ptx::pack_bf16(a2, a3));
        }
        // lane (g, t): depths g * D/8 .. + D/8 of keys 2t, 2t+1, 2t+8, 2t+9
        constexpr int VW = C::FP4 ? D / 64 : D / 32;
        uint32_t v[4][VW];
        uint32_t s01 = 0u, s23 = 0u;   // e2m1: block scales of the keys' depths, as f16
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + C::key_row(2 * t + (e & 1)) + 8 * (e >> 1);
          const uint32_t at = st + C::KV + row * C::ROWB;
          if constexpr (C::FP4) {
            if constexpr (D == 128) {
              const uint2 w = ptx::ld_shared_v2(at + C::swz_v(row, g >> 1) * 16 + (g & 1) * 8);
              v[e][0] = w.x; v[e][1] = w.y;
            } else {
              v[e][0] = ptx::ld_shared_u32(at + 4 * g);
            }
            const uint32_t b =
                ptx::ld_shared_u8(st + 2 * (C::KV + C::SC) + C::BL + row * C::BK + (D == 128 ? g : g >> 1)) << (8 * (e & 1));
            if (e < 2) s01 |= b;
            else s23 |= b;
          } else if constexpr (D == 128) {
            const uint4 w = ptx::ld_shared_v4(at + C::swz_v(row, g) * 16);
            v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
          } else {
            const uint2 w = ptx::ld_shared_v2(at + C::swz_v(row, g >> 1) * 16 + (g & 1) * 8);
            v[e][0] = w.x; v[e][1] = w.y;
          }
        }
        if constexpr (C::FP4) {
          s01 = ptx::e4m3x2_to_f16x2(s01);
          s23 = ptx::e4m3x2_to_f16x2(s23);
        }
        // (key, key) pairs of each depth
        auto product4 = [&](auto f16) {
          constexpr uint32_t LOW = 0x0f0f0f0fu;
#pragma unroll
          for (int w = 0; w < VW; ++w) {
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
        };
        auto product = [&](auto f16) {
          if constexpr (C::FP4) {
            product4(f16);
            return;
          }
          if constexpr (!C::FP4) {
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140);
              const uint32_t hi = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
              uint32_t a[4];
              if constexpr (decltype(f16)::value) {
                ptx::e4m3x4_to_f16x2(lo, a[0], a[1]);
                ptx::e4m3x4_to_f16x2(hi, a[2], a[3]);
#pragma unroll
                for (int x = 0; x < NT; ++x) ptx::mma_16816_f16(acc[2 * w + h][x], a, pf[x][0], pf[x][1]);
              } else {
                a[0] = ptx::e4m3x2_to_bf16x2(lo & 0xffffu);
                a[1] = ptx::e4m3x2_to_bf16x2(lo >> 16);
                a[2] = ptx::e4m3x2_to_bf16x2(hi & 0xffffu);
                a[3] = ptx::e4m3x2_to_bf16x2(hi >> 16);
#pragma unroll
                for (int x = 0; x < NT; ++x) ptx::mma_16816(acc[2 * w + h][x], a, pf[x][0], pf[x][1]);
              }
            }
          }
        };
        if (as_f16) product(std::true_type{});
        else product(std::false_type{});
      }
    }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[x][e] += __shfl_xor_sync(kFull, l[x][e], o);

  if constexpr (C::CODES) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][x][e] *= vref * 0.0078125f;
  }

  if (first + pc.count < end) {
    next = walk.at(P, first + pc.count, end, next_rows);
    load_q<C>(P, next, next_rows, qf);
  }

  // ---- The key groups' results meet in shared memory, each group's in the
  // stage it used last (the loader does not fill that one before the next
  // piece's first tile). Without keys there is no such stage, and only the
  // (maximum, sum) say so.
  float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);   // [WK][RT]
  const int last = ((count + C::STAGES - 1) % C::STAGES) * C::STAGE;
  group_sync();   // the group is done with its last tile
  if (n > 0) {
    float* part = reinterpret_cast<float*>(smem + C::part_at(kg, last));   // [RT][D]
#pragma unroll
    for (int x = 0; x < NT; ++x)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 8 * (NT * wm + x) + 2 * t + e;
        float* dst = part + r * D;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          if constexpr (C::CODES) {
            *reinterpret_cast<float2*>(dst + C::part_col(r, g * (D / 8) + 2 * i)) = make_float2(acc[i][x][e], acc[i][x][2 + e]);
          } else {
            dst[C::part_col(r, 16 * i + g)] = acc[i][x][e];
            dst[C::part_col(r, 16 * i + g + 8)] = acc[i][x][2 + e];
          }
        }
      }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (g == 0) ml[kg * C::RT + 8 * (NT * wm + x) + 2 * t + e] = make_float2(m[x][e], l[x][e]);
  __syncthreads();
  auto finish_row = [&](int, int row, int d, const float4& o, float mm, float ll) {
    const RowAt a = row_at(P, hk, rt * C::RT + row);
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    *reinterpret_cast<uint2*>(o_at(P, s, pc.b, a) + d) =
        make_uint2(ptx::pack_bf16(o.x * inv, o.y * inv), ptx::pack_bf16(o.z * inv, o.w * inv));
    if (d == 0 && P.lse != nullptr) P.lse[lse_at(P, s, pc.b, a)] = lse_of(mm, ll);
  };
  auto keep_row = [&](int64_t slot, int row, int d, const float4& o, float mm, float ll) {
    *reinterpret_cast<float4*>(P.part_o + (slot * C::RT + row) * D + d) = o;
    if (d == 0) P.part_ml[slot * C::RT + row] = make_float2(mm, ll);
  };
  const bool whole = pc.count == pc.tiles;
  const int valid = min(C::RT, rows - rt * C::RT);
  const int64_t mine = 2 * (int64_t)blockIdx.x + (pc.first == 0 ? 1 : 0);
  for (int x = threadIdx.x; x < valid * (D / 4); x += kThreads) {
    const int row = x / (D / 4), d = 4 * (x % (D / 4));
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < C::WK; ++k) mm = fmaxf(mm, ml[k * C::RT + row].x);
    const float base = mm == -INFINITY ? 0.f : mm;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C::WK; ++k) {
      const float2 kml = ml[k * C::RT + row];
      const float w = ptx::ex2(kml.x - base);
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (n > 0)
        v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + C::part_at(k, last)) + row * D +
                                             C::part_col(row, d));
      ll = fmaf(w, kml.y, ll);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    if (whole) finish_row(0, row, d, o, mm, ll);
    else keep_row(mine, row, d, o, mm, ll);
  }
  if (whole) {
    __syncthreads();   // before the next piece loads over the parts
    return;
  }
  const int start = first - pc.first, c0 = start / per, parts = (start + pc.tiles - 1) / per - c0 + 1;
  const int hood = ((int)blockIdx.x / P.team - c0) / kJoin, in_hood = min(kJoin, parts - kJoin * hood);
  const int hoods = (parts + kJoin - 1) / kJoin;
  // counters: [0] a segment's first neighbourhood by its first CTA, [1] others
  // by theirs, [2] neighbourhoods by the segment's first CTA
  uint32_t* const counters = P.counters;
  const int grid = gridDim.x;
  auto slot_in_hood = [&](int i) { return 2 * (int64_t)cta_of(P, c0 + kJoin * hood + i) + (hood == 0 && i == 0 ? 1 : 0); };
  if (!count_in(counters + (hood == 0 ? 0 : grid) + cta_of(P, c0 + kJoin * hood), in_hood)) return;
  if (hoods == 1) {
    join_parts<C>(P, in_hood, valid, slot_in_hood, finish_row);
    return;
  }
  // The joined part overwrites the first one's: every thread its own columns,
  // but the (maximum, sum) of a row only once all threads have read them.
  float2 kept[C::ROUNDS];
#pragma unroll
  for (int i = 0; i < C::ROUNDS; ++i) kept[i] = make_float2(0.f, 0.f);
  join_parts<C>(P, in_hood, valid, slot_in_hood, [&](int round, int row, int d, const float4& o, float mm, float ll) {
    *reinterpret_cast<float4*>(P.part_o + (slot_in_hood(0) * C::RT + row) * D + d) = o;
    kept[round] = make_float2(mm, ll);
  });
  __syncthreads();
#pragma unroll
  for (int i = 0; i < C::ROUNDS; ++i) {
    const int x = threadIdx.x + i * kThreads;
    if (x < valid * (D / 4) && x % (D / 4) == 0) P.part_ml[slot_in_hood(0) * C::RT + x / (D / 4)] = kept[i];
  }
  if (!count_in(counters + 2 * grid + cta_of(P, c0), hoods)) return;
  join_parts<C>(P, hoods, valid, [&](int i) { return 2 * (int64_t)cta_of(P, c0 + kJoin * i) + (i == 0 ? 1 : 0); }, finish_row);
}

template <int D, int KIND, int NT, int WM>
__global__ void __launch_bounds__(kThreads, (Cfg<D, KIND, NT, WM>::CTAS))
    paged_stream_kernel(const __grid_constant__ StreamParams P) {
  using C = Cfg<D, KIND, NT, WM>;
  extern __shared__ __align__(128) uint8_t smem[];
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  Loader<C> load;
  const int total = load.walk.start(P);
  const int teams = (int)gridDim.x / P.team;
  const int per = (total + teams - 1) / teams;
  int x = min(total, (int)blockIdx.x / P.team * per);
  const int end = min(total, x + per);
  if (x >= end) return;
  // Fill the ring, then run the pieces; the loader stays STAGES - 1 tiles ahead.
  const int warp = threadIdx.x >> 5, kg = warp / C::WM, gt = (warp % C::WM) * 32 + (threadIdx.x & 31);
  const uint32_t ring = ptx::smem_u32(smem) + kg * (C::STAGES * C::STAGE);
  if (P.s.batch > 32) load.walk.seek(P, x);
  Walker<C> walk = load.walk;
  SeqRows s;
  Piece pc = walk.at(P, x, end, s);
  uint32_t qf[C::NT][D / 16][2];
  load_q<C>(P, pc, s, qf);
  load.x = x;
  load.end = end;
  load.next_piece(P, gt, kg);
#pragma unroll 1
  for (int j = 0; j < C::STAGES - 1; ++j) {
    load.issue(P, ring + j * C::STAGE, gt, kg);
    ptx::cp_async_commit();
  }
  int count = 0;   // tiles used so far
  while (x < end && pc.count > 0) {
    Piece next = pc;
    SeqRows next_rows = s;
    run_piece<C>(P, pc, s, smem, load, walk, qf, next, next_rows, count, x, end, per);
    x += pc.count;
    pc = next;
    s = next_rows;
  }
  ptx::cp_async_wait<0>();
}

template <int D, int KIND, int NT, int WM>
cudaError_t launch_t(const StreamParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, KIND, NT, WM>;
  constexpr auto kern = paged_stream_kernel<D, KIND, NT, WM>;
  return launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), kThreads, C::SMEM, stream); });
}

template <int D, int KIND>
cudaError_t launch_d(const StreamParams& p, int row_tile, int grid, cudaStream_t stream) {
  switch (row_tile) {
    case 8: return launch_t<D, KIND, 1, 1>(p, grid, stream);
    case 16: return launch_t<D, KIND, 2, 1>(p, grid, stream);
    default: return launch_t<D, KIND, 2, 2>(p, grid, stream);
  }
}

template <int D>
cudaError_t launch_k(const StreamParams& p, int kind, int row_tile, int grid, cudaStream_t stream) {
  return kind == kBf16 ? launch_d<D, kBf16>(p, row_tile, grid, stream)
                       : (kind == kE4m3 ? launch_d<D, kE4m3>(p, row_tile, grid, stream)
                                        : launch_d<D, kE2m1>(p, row_tile, grid, stream));
}

}  // namespace

cudaError_t paged_stream_launch(const StreamParams& p, int head_dim, int kind, int row_tile, int grid,
                                cudaStream_t stream) {
  return head_dim == 128 ? launch_k<128>(p, kind, row_tile, grid, stream) : launch_k<64>(p, kind, row_tile, grid, stream);
}

}  // namespace af
