// What the streaming attention kernels (paged_stream.cu, paged_stream4.cu) share:
// how a CTA finds its part of the work, and how the parts of a segment are joined.
//
// C, a kernel's configuration, has D, RT (rows of a row tile), TILE (keys of a
// unit of work), WK (key groups of a CTA), NT and WM (8-row tiles of a warp, warps
// of a key group), part_col and q_depth; and the FT threads that finish a piece:
// their number among them, ftid(), and barrier, fsync().
#pragma once
#include <math.h>
#include <stdint.h>

#include "paged.h"
#include "ptx.cuh"

namespace af {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int min_int(int a, int b) { return a < b ? a : b; }

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
// counter at zero). `counted`: thread 0 has done so already, being the n-th from 0.
template <class C>
__device__ __forceinline__ bool count_in(uint32_t* counter, uint32_t want, bool counted = false, uint32_t n = 0u) {
  __shared__ bool is_last;
  C::fsync();
  if (C::ftid() == 0) {
    if (!counted) {
      __threadfence();   // (of the whole CTA's stores: the barrier above orders them before it)
      n = atomicAdd(counter, 1u);
    }
    is_last = n == want - 1u;
    if (is_last) *counter = 0u;
    __threadfence();
  }
  C::fsync();
  return is_last;
}
// Which of a segment's parts a CTA has, the piece's first unit being `first` among all
// and `per` the units of every CTA: the parts, from team c0 on, this one's neighbourhood,
// how many are in there, and neighbourhoods.
struct PartOf {
  int c0, parts, hood, in_hood, hoods;
  __device__ __forceinline__ PartOf(const StreamParams& P, const Piece& pc, int first, int per) {
    const int start = first - pc.first;
    c0 = start / per;
    parts = (start + pc.tiles - 1) / per - c0 + 1;
    hood = ((int)blockIdx.x / P.team - c0) / kJoin;
    in_hood = min(kJoin, parts - kJoin * hood);
    hoods = (parts + kJoin - 1) / kJoin;
  }
  // Counters: [0] a segment's first neighbourhood by its first CTA, [1] others by theirs,
  // [2] neighbourhoods by the segment's first CTA.
  __device__ __forceinline__ uint32_t* counter(const StreamParams& P) const {
    return P.counters + (hood == 0 ? 0 : (int)gridDim.x) + cta_of(P, c0 + kJoin * hood);
  }
};

// 16-byte pieces of a row tile per thread.
template <class C>
constexpr int rounds() { return (C::RT * (C::D / 4) + C::FT - 1) / C::FT; }

// Sums parts 0 .. n - 1 at slots slot(i) of the segment's `valid` rows; hands
// (round, row, depth, four sums, maximum, sum) to `put`, whose thread alone
// holds them (round: of this thread's, a constant after unrolling). Sixteen
// loads of a thread are in flight: up to four rows, times parts. ROLLED: `round` need
// not be a constant.
template <class C, bool ROLLED, class Slot, class Put>
__device__ __forceinline__ void join_parts(const StreamParams& P, int n, int valid, Slot slot, Put put) {
  constexpr int D = C::D, ROUNDS = rounds<C>(), IT = min_int(ROUNDS, 4), PB = 16 / IT;
#pragma unroll (ROLLED ? 1 : ROUNDS / IT)
  for (int g = 0; g < ROUNDS / IT; ++g) {
    float mm[IT], ll[IT];
    float4 o[IT];
#pragma unroll
    for (int y = 0; y < IT; ++y) {
      mm[y] = -INFINITY;
      ll[y] = 0.f;
      o[y] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const int x0 = C::ftid() + g * IT * C::FT;
    if (x0 >= valid * (D / 4)) break;
    for (int i0 = 0; i0 < n; i0 += PB) {
      float4 v[IT][PB];
      float2 ml[IT][PB];
#pragma unroll
      for (int i = 0; i < PB; ++i)
#pragma unroll
        for (int y = 0; y < IT; ++y) {
          const int x = x0 + y * C::FT;
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
      const int x = x0 + y * C::FT;
      if (x < valid * (D / 4)) put(g * IT + y, x / (D / 4), 4 * (x % (D / 4)), o[y], mm[y], ll[y]);
    }
  }
}

// q of a piece's rows, for warp wm of a key group: row g of each of its column tiles,
// pairs at depths d and d + step of every 16. The loads stay where they are written.
template <class C>
__device__ __forceinline__ void load_q(const StreamParams& P, const Piece& pc, const SeqRows& s, int wm,
                                       uint32_t (&qf)[C::NT][C::D / 16][2]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int row0 = row_tile_of(P, pc.seg) * C::RT + 8 * C::NT * wm;
#pragma unroll
  for (int x = 0; x < C::NT; ++x) {
    const int r = row0 + 8 * x + g;
    const bool ok = r < s.lq * P.group;
    const uint8_t* src = q_row(P, s, pc.b, row_at(P, head_of(P, pc.seg), ok ? r : 0));
#pragma unroll
    for (int kk = 0; kk < C::D / 16; ++kk) {
      const int d = C::q_depth(kk, t);
      const int step = C::Q_STEP;
      qf[x][kk][0] = ok ? (uint32_t)ptx::ld_global_pinned(reinterpret_cast<const int*>(src + 2 * d)) : 0u;
      qf[x][kk][1] = ok ? (uint32_t)ptx::ld_global_pinned(reinterpret_cast<const int*>(src + 2 * (d + step))) : 0u;
    }
  }
}

// Writes the row piece (row, d .. d + 3) of a segment: its sums over l, and lse.
template <class C>
__device__ __forceinline__ void finish_row(const StreamParams& P, const Piece& pc, const SeqRows& s, int row, int d,
                                           const float4& o, float mm, float ll) {
  const RowAt a = row_at(P, head_of(P, pc.seg), row_tile_of(P, pc.seg) * C::RT + row);
  const float inv = ll == 0.f ? 0.f : 1.f / ll;
  *reinterpret_cast<uint2*>(o_at(P, s, pc.b, a) + d) =
      make_uint2(ptx::pack_bf16(o.x * inv, o.y * inv), ptx::pack_bf16(o.z * inv, o.w * inv));
  if (d == 0 && P.lse != nullptr) P.lse[lse_at(P, s, pc.b, a)] = lse_of(mm, ll);
}
template <class C>
__device__ __forceinline__ int rows_of_piece(const StreamParams& P, const Piece& pc, const SeqRows& s) {
  return min(C::RT, s.lq * P.group - row_tile_of(P, pc.seg) * C::RT);
}

// Sums the key groups of a piece, whose results have been left in shared memory
// (a barrier ago): `ml` [WK][RT] maxima and sums, part(k) group k's [RT][D]
// accumulators, or NULL where it had no keys. Rows of a segment that lies in this
// CTA are written, others left as a part of it.
template <class C, class Part>
__device__ __forceinline__ void leave_piece(const StreamParams& P, const Piece& pc, const SeqRows& s, const float2* ml,
                                            Part part) {
  constexpr int D = C::D;
  const bool whole = pc.count == pc.tiles;
  const int valid = rows_of_piece<C>(P, pc, s);
  const int64_t mine = 2 * (int64_t)blockIdx.x + (pc.first == 0 ? 1 : 0);
  for (int x = C::ftid(); x < valid * (D / 4); x += C::FT) {
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
      if (const float* from = part(k); from != nullptr)
        v = *reinterpret_cast<const float4*>(from + row * D + C::part_col(row, d));
      ll = fmaf(w, kml.y, ll);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    if (whole) {
      finish_row<C>(P, pc, s, row, d, o, mm, ll);
    } else {
      *reinterpret_cast<float4*>(P.part_o + (mine * C::RT + row) * D + d) = o;
      if (d == 0) P.part_ml[mine * C::RT + row] = make_float2(mm, ll);
    }
  }
}

// Joins the parts of a piece's segment if this CTA is the last to count itself in
// (`counted`, `n`: as count_in).
template <class C>
__device__ __forceinline__ void join_piece(const StreamParams& P, const Piece& pc, const SeqRows& s, int first, int per,
                                           bool counted = false, uint32_t n = 0u) {
  constexpr int D = C::D;
  const int valid = rows_of_piece<C>(P, pc, s);
  const PartOf at(P, pc, first, per);
  const int c0 = at.c0, hood = at.hood, in_hood = at.in_hood, hoods = at.hoods;
  auto finish = [&](int, int row, int d, const float4& o, float mm, float ll) { finish_row<C>(P, pc, s, row, d, o, mm, ll); };
  auto slot_in_hood = [&](int i) { return 2 * (int64_t)cta_of(P, c0 + kJoin * hood + i) + (hood == 0 && i == 0 ? 1 : 0); };
  if (!count_in<C>(at.counter(P), in_hood, counted, n)) return;
  if (hoods == 1) {
    join_parts<C, true>(P, in_hood, valid, slot_in_hood, finish);
    return;
  }
  // The joined part overwrites the first one's: every thread its own columns,
  // but the (maximum, sum) of a row only once all threads have read them.
  float2 kept[rounds<C>()];
#pragma unroll
  for (int i = 0; i < rounds<C>(); ++i) kept[i] = make_float2(0.f, 0.f);
  join_parts<C, false>(P, in_hood, valid, slot_in_hood, [&](int round, int row, int d, const float4& o, float mm, float ll) {
    *reinterpret_cast<float4*>(P.part_o + (slot_in_hood(0) * C::RT + row) * D + d) = o;
    kept[round] = make_float2(mm, ll);
  });
  C::fsync();
#pragma unroll
  for (int i = 0; i < rounds<C>(); ++i) {
    const int x = C::ftid() + i * C::FT;
    if (x < valid * (D / 4) && x % (D / 4) == 0) P.part_ml[slot_in_hood(0) * C::RT + x / (D / 4)] = kept[i];
  }
  if (!count_in<C>(P.counters + 2 * (int)gridDim.x + cta_of(P, c0), hoods)) return;
  join_parts<C, true>(P, hoods, valid, [&](int i) { return 2 * (int64_t)cta_of(P, c0 + kJoin * i) + (i == 0 ? 1 : 0); }, finish);
}

// Both: rows of a segment of several CTAs are finished by whichever comes last.
template <class C, class Part>
__device__ __forceinline__ void finish_piece(const StreamParams& P, const Piece& pc, const SeqRows& s, const float2* ml,
                                             Part part, int first, int per) {
  leave_piece<C>(P, pc, s, ml, part);
  if (pc.count == pc.tiles) C::fsync();   // before the next piece loads over the parts
  else join_piece<C>(P, pc, s, first, per);
}

}  // namespace af
