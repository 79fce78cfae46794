// Attention of a few new tokens over the paged cache: a streaming kernel for
// problems that HBM bounds, and the merge of its partial results.
//
// The new tokens of one sequence times the query heads that share one KV head
// are R = Lq * Hq / Hkv rows over the same keys. For few rows the cached K and V
// are all that matters: they have to cross HBM once, and R flops per byte leave
// the tensor cores idle. So the kernel is built around the loads:
//   * the work is the list of all 64-key tiles of all (sequence, KV head, row
//     tile) segments, cut into equal contiguous parts, one per CTA (two CTAs per
//     SM). Lengths are read on the device, so ragged batches balance without the
//     host knowing them and a captured call follows lengths that change;
//   * a CTA streams its tiles through a ring of cp.async stages (about 96 KB in
//     flight per CTA). A row tile is 16 * WM rows (WM = 1, 2, 4); the four warps
//     form 4 / WM key groups of WM warps, each group with its own keys and ring,
//     so with up to 16 rows every warp streams by itself and no barrier is met
//     inside a segment;
//   * one pass with running maximum and sum (fp32, log2 units), m16n8k16 tensor
//     instructions: the rows are too few for the 128-row instructions of the
//     tcgen05 kernel, and the loads bound both. The maximum only moves when it
//     grows by more than 2^8, so the accumulator is rarely rescaled; O and the
//     sum share it, so their quotient is exact;
//   * an e4m3 cache is widened to bf16 in registers (exactly; the key scale is
//     applied to the fp32 score, the value scale to the fp32 weight before its
//     rounding to bf16). Depth and value columns are dealt to lanes in the order
//     in which 16-byte reads from shared memory deliver them: a dot product does
//     not depend on the order of its depth, nor a product on that of its columns;
//   * a segment that lies in one CTA is finished there; the others leave their
//     accumulator, maximum and sum in the workspace (at most two per CTA) and a
//     second small kernel, already resident when the first one ends, merges them.
// Slots at or past the sequence's end are not read (their shared memory is
// zeroed), so whatever they hold cannot reach a result.
#include <math.h>

#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"

namespace af {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kThreads = 128;
constexpr int min_int(int a, int b) { return a < b ? a : b; }

// NT * 8 rows per warp, WM warps to a key group.
template <int D_, bool FP8_, int NT_, int WM_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WM = WM_;
  static constexpr bool FP8 = FP8_;
  static constexpr int WK = 4 / WM;              // key groups
  static constexpr int RT = 8 * NT * WM;         // rows of a row tile
  static constexpr int ROWB = FP8 ? D : 2 * D;   // bytes of a cached row
  static constexpr int KW = stream_tile(ROWB, WM) / WK;   // keys of a group per tile
  static constexpr int TILE = KW * WK;
  static constexpr int BLOCKS = KW / 16;         // 16-key blocks of a group's tile
  static constexpr int CPR = ROWB / 16;          // 16-byte pieces of a row
  static constexpr int GT = 32 * WM;             // threads of a group
  static constexpr int RS = GT / CPR;            // rows a group loads at a time
  static constexpr int NL = KW / RS;             // loads per thread of K (and of V)
  static constexpr int KV = KW * ROWB;
  static constexpr int SC = FP8 ? KW * 4 : 0;
  static constexpr int STAGE = 2 * KV + 2 * SC;  // bytes of one group's stage
  static constexpr int STAGES = min_int(8, 98304 / (WK * 2 * KV));
  static constexpr int PITCH = D + 8;            // floats of a row in the group merge
  static constexpr int RING = WK * STAGES * STAGE;
  static constexpr int MERGE = WK * RT * (PITCH + 2) * 4;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;   // the merge reuses the ring
  static_assert(STAGES >= 3 && SMEM <= 113 * 1024, "two CTAs per SM");
  // Position of 16-byte piece `c` of row `r` in a stage (bank conflicts).
  __device__ static int swz_k(int r, int c) {
    return FP8 ? (CPR == 8 ? c ^ ((r & 1) << 2) : c) : c ^ (r & 7);
  }
  __device__ static int swz_v(int r, int c) { return FP8 && CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); }
};

// Work units of sequence b: row tiles * KV heads * (key tiles, or 1 unsplit).
struct SeqUnits {
  SeqRows r;
  int row_tiles, tiles, units;
};

template <class C>
__device__ __forceinline__ SeqUnits seq_units(const StreamParams& P, int b) {
  SeqUnits u;
  u.r = load_seq(P.s, b, P.ws);
  u.row_tiles = (int)(((int64_t)u.r.lq * P.group + C::RT - 1) / C::RT);
  u.tiles = P.split ? max(1, (u.r.lk + C::TILE - 1) / C::TILE) : 1;
  u.units = u.row_tiles * P.c.heads_kv * u.tiles;
  return u;
}

// One contiguous part of a segment.
struct Piece {
  int b, seg;            // seg = row tile * Hkv + KV head
  int first, count;      // unit range within the segment
  int tiles;             // units of the segment
};

template <class C>
struct Walker {
  int b = 0;             // first sequence of the current window of 32
  int base = 0;          // units in front of it
  // Piece that holds unit x, cut at `end`. All lanes of the warp; x increases.
  __device__ __forceinline__ Piece at(const StreamParams& P, int x, int end, SeqRows& rows) {
    const int lane = threadIdx.x & 31;
    while (true) {
      SeqUnits u;
      u.units = 0;
      if (b + lane < P.s.batch) u = seq_units<C>(P, b + lane);
      int incl = u.units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += n;
      }
      const unsigned hit = __ballot_sync(kFull, b + lane < P.s.batch && x < base + incl);
      if (hit) {
        const int w = __ffs(hit) - 1;
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
      base += __shfl_sync(kFull, incl, 31);
      b += 32;
      if (b >= P.s.batch) {   // cannot happen while x < total
        Piece p = {0, 0, 0, 0, 1};
        rows = {0, 0, 0};
        return p;
      }
    }
  }
};

template <class C>
__device__ __forceinline__ int total_units(const StreamParams& P) {
  int n = 0;
  for (int b = threadIdx.x & 31; b < P.s.batch; b += 32) n += seq_units<C>(P, b).units;
  return __reduce_add_sync(kFull, n);
}

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

template <class C>
__device__ void run_piece(const StreamParams& P, const Piece& pc, const SeqRows& s, uint8_t* smem) {
  constexpr int D = C::D, WM = C::WM, NT = C::NT, KW = C::KW, NB = C::BLOCKS;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int wm = warp % WM, kg = warp / WM;
  const int gt = wm * 32 + lane;                  // thread within its key group
  const int hk = pc.seg % P.c.heads_kv, rt = pc.seg / P.c.heads_kv;
  const int rows = s.lq * P.group;
  const uint32_t ring = ptx::smem_u32(smem) + kg * (C::STAGES * C::STAGE);
  const int key_tiles = (s.lk + C::TILE - 1) / C::TILE;
  const int t0 = P.split ? pc.first : 0;
  const int n = P.split ? min(pc.count, key_tiles - t0) : key_tiles;
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
  // q of row g of each column tile: pairs at depths d and d + step of every 16
  uint32_t qf[NT][D / 16][2];
#pragma unroll
  for (int x = 0; x < NT; ++x) {
    const int r = row0 + 8 * x + g;
    const bool ok = r < rows;
    const RowAt a = row_at(P, hk, ok ? r : 0);
    const uint8_t* src = P.q + (P.s.cu_q != nullptr ? 0 : pc.b * P.q_b) + (int64_t)(s.q0 + a.i) * P.q_t + a.h * P.q_h;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int d = C::FP8 ? 16 * (t + 4 * (kk >> 2)) + 4 * (kk & 3) : 16 * kk + 2 * t;
      const int step = C::FP8 ? 2 : 8;
      qf[x][kk][0] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 2 * d)) : 0u;
      qf[x][kk][1] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 2 * (d + step))) : 0u;
    }
    if constexpr (C::FP8) {
      // The codes of an e4m3 cache are multiplied as f16 (one conversion for two
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

  const uint8_t* kbase = P.c.k + hk * P.c.k_head;
  const uint8_t* vbase = P.c.v + hk * P.c.v_head;
  const int page_mask = (1 << P.c.page_shift) - 1;
  const int lrow = gt / C::CPR, lcol = gt % C::CPR;

  // Pages of the 16-key blocks of a group's tile, fetched one tile ahead of
  // their use (the loads' addresses depend on them).
  int pages[NB];
  auto fetch_pages = [&](int j) {
    const int key0 = (t0 + j) * C::TILE + kg * KW;
#pragma unroll
    for (int u = 0; u < NB; ++u)
      pages[u] = (j < n && key0 + 16 * u < s.lk) ? load_page(P.c, pc.b, (key0 + 16 * u) >> P.c.page_shift, P.ws) : 0;
  };
  auto load_tile = [&](int j) {
    const int key0 = (t0 + j) * C::TILE + kg * KW;
    const uint32_t st = ring + (j % C::STAGES) * C::STAGE;
    constexpr int PER = C::RS <= 16 ? 16 / C::RS : 1;   // loads of a 16-key block per thread
#pragma unroll
    for (int i = 0; i < C::NL; i += PER) {
      // block of these loads' rows (RS = 32: of this thread's row)
      const int u = C::RS <= 16 ? i / PER : 2 * i;
      const int page = C::RS <= 16 || lrow < 16 ? pages[u] : pages[u + (C::RS > 16 ? 1 : 0)];
      const int64_t slot = (key0 + lrow + i * C::RS) & page_mask;
      const uint8_t* ks = kbase + page * P.c.k_page + slot * P.c.k_tok + lcol * 16;
      const uint8_t* vs = vbase + page * P.c.v_page + slot * P.c.v_tok + lcol * 16;
#pragma unroll
      for (int x = 0; x < PER; ++x) {
        const int row = lrow + (i + x) * C::RS;
        const bool ok = key0 + row < s.lk;
        ptx::cp_async16(st + row * C::ROWB + C::swz_k(row, lcol) * 16, ok ? ks : P.c.k, ok);
        ptx::cp_async16(st + C::KV + row * C::ROWB + C::swz_v(row, lcol) * 16, ok ? vs : P.c.v, ok);
        ks += C::RS * P.c.k_tok;
        vs += C::RS * P.c.v_tok;
      }
    }
    if constexpr (C::FP8) {
      // scales: 4 keys per 16 bytes; a piece that crosses the end is cut there
      if (gt < 2 * KW / 4) {
        const int which = gt / (KW / 4), k4 = 4 * (gt % (KW / 4));
        int page = pages[0];
#pragma unroll
        for (int u = 1; u < NB; ++u)
          if ((k4 >> 4) == u) page = pages[u];
        const int left = s.lk - (key0 + k4);
        const int bytes = left >= 4 ? 16 : (left > 0 ? 4 * left : 0);
        const float* base = which ? P.c.v_scale : P.c.k_scale;
        const float* src =
            bytes ? base + ((((int64_t)page * P.c.heads_kv + hk) << P.c.page_shift) + ((key0 + k4) & page_mask)) : base;
        const uint32_t dst = st + 2 * C::KV + which * C::SC + k4 * 4;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
      }
    }
  };
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
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[x][e] = -INFINITY;
      l[x][e] = 0.f;
    }

  fetch_pages(0);
#pragma unroll 1
  for (int j = 0; j < C::STAGES - 1; ++j) {
    if (j < n) load_tile(j);
    ptx::cp_async_commit();
    fetch_pages(j + 1);
  }
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    ptx::cp_async_wait<C::STAGES - 2>();
    group_sync();   // tile j has arrived, and nobody reads tile j - 1's stage any more
    if (j + C::STAGES - 1 < n) load_tile(j + C::STAGES - 1);
    ptx::cp_async_commit();
    fetch_pages(j + C::STAGES);

    const uint32_t st = ring + (j % C::STAGES) * C::STAGE;
    const int key0 = (t0 + j) * C::TILE + kg * KW;
    // ---- S^T = K Q^T: keys g and g + 8 of each block by rows 2 t, 2 t + 1 of each column tile
    float sc[NB][NT][4];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[i][x][e] = 0.f;
    if constexpr (!C::FP8) {
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
      if constexpr (C::FP8) {
        k0 = scale_sm[16 * i + g];
        k1 = scale_sm[16 * i + g + 8];
      }
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[i][x][e] *= C::FP8 ? qscale[x][e & 1] * (e < 2 ? k0 : k1) : qscale[x][e & 1];
    }
    if (key0 + KW > lim_min) {
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int x = 0; x < NT; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (key0 + 16 * i + g + 8 * (e >> 1) >= lim[x][e & 1]) sc[i][x][e] = -INFINITY;
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
    // ---- weights (a row that has seen no key yet keeps m = -inf and weights 0), O^T += V^T P^T
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      uint32_t pf[NT][2];
      float v0 = 1.f, v1 = 1.f;
      if constexpr (C::FP8) {
        v0 = scale_sm[KW + 16 * i + g];
        v1 = scale_sm[KW + 16 * i + g + 8];
      }
#pragma unroll
      for (int x = 0; x < NT; ++x) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float off = m[x][e & 1] == -INFINITY ? 0.f : m[x][e & 1];
          w[e] = ptx::ex2(sc[i][x][e] - off);
          l[x][e & 1] += w[e];
          if constexpr (C::FP8) w[e] *= e < 2 ? v0 : v1;
        }
        // (key, rows) pairs to (row, keys) pairs
        pf[x][0] = ptx::movmatrix_trans(ptx::pack_bf16(w[0], w[1]));
        pf[x][1] = ptx::movmatrix_trans(ptx::pack_bf16(w[2], w[3]));
      }
      if constexpr (!C::FP8) {
#pragma unroll
        for (int q = 0; q < D / 16; ++q) {
          uint32_t a[4];
          const int row = 16 * i + (lane & 7) + 8 * (lane >> 4);
          ptx::ldmatrix_x4_trans(st + C::KV + row * C::ROWB + C::swz_v(row, 2 * q + ((lane >> 3) & 1)) * 16, a);
#pragma unroll
          for (int x = 0; x < NT; ++x) ptx::mma_16816(acc[q][x], a, pf[x][0], pf[x][1]);
        }
      } else {
        // lane (g, t): depths g * D/8 .. + D/8 of keys 2t, 2t+1, 2t+8, 2t+9
        uint32_t v[4][D / 32];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * i + 2 * t + (e & 1) + 8 * (e >> 1);
          const uint32_t at = st + C::KV + row * C::ROWB;
          if constexpr (D == 128) {
            const uint4 w = ptx::ld_shared_v4(at + C::swz_v(row, g) * 16);
            v[e][0] = w.x; v[e][1] = w.y; v[e][2] = w.z; v[e][3] = w.w;
          } else {
            const uint2 w = ptx::ld_shared_v2(at + C::swz_v(row, g >> 1) * 16 + (g & 1) * 8);
            v[e][0] = w.x; v[e][1] = w.y;
          }
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t lo = __byte_perm(v[0][w], v[1][w], h ? 0x7362 : 0x5140);
            const uint32_t hi = __byte_perm(v[2][w], v[3][w], h ? 0x7362 : 0x5140);
            const uint32_t a[4] = {ptx::e4m3x2_to_bf16x2(lo & 0xffffu), ptx::e4m3x2_to_bf16x2(lo >> 16),
                                   ptx::e4m3x2_to_bf16x2(hi & 0xffffu), ptx::e4m3x2_to_bf16x2(hi >> 16)};
#pragma unroll
            for (int x = 0; x < NT; ++x) ptx::mma_16816(acc[2 * w + h][x], a, pf[x][0], pf[x][1]);
          }
        }
      }
    }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[x][e] += __shfl_xor_sync(kFull, l[x][e], o);
  ptx::cp_async_wait<0>();

  // ---- the key groups' results meet in shared memory (over the ring)
  float* buf = reinterpret_cast<float*>(smem);                          // [WK][RT][PITCH]
  float2* ml = reinterpret_cast<float2*>(buf + C::WK * C::RT * C::PITCH);   // [WK][RT]
  __syncthreads();
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = kg * C::RT + 8 * (NT * wm + x) + 2 * t + e;
      float* dst = buf + r * C::PITCH;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        if constexpr (C::FP8) {
          *reinterpret_cast<float2*>(dst + g * (D / 8) + 2 * i) = make_float2(acc[i][x][e], acc[i][x][2 + e]);
        } else {
          dst[16 * i + g] = acc[i][x][e];
          dst[16 * i + g + 8] = acc[i][x][2 + e];
        }
      }
      if (g == 0) ml[r] = make_float2(m[x][e], l[x][e]);
    }
  __syncthreads();
  const bool whole = pc.count == pc.tiles;
  // a part of a segment: slot 2c if it continues an earlier CTA's, 2c + 1 if it starts one
  const int64_t slot = ((int64_t)2 * blockIdx.x + (pc.first == 0 ? 1 : 0)) * C::RT;
  for (int x = threadIdx.x; x < C::RT * (D / 4); x += kThreads) {
    const int row = x / (D / 4), d = 4 * (x % (D / 4));
    const int r = rt * C::RT + row;
    if (r >= rows) break;
    float mm = -INFINITY, ll = 0.f;
#pragma unroll
    for (int k = 0; k < C::WK; ++k) mm = fmaxf(mm, ml[k * C::RT + row].x);
    const float base = mm == -INFINITY ? 0.f : mm;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C::WK; ++k) {
      const float2 kml = ml[k * C::RT + row];
      const float w = ptx::ex2(kml.x - base);
      const float4 v = *reinterpret_cast<const float4*>(buf + (k * C::RT + row) * C::PITCH + d);
      ll = fmaf(w, kml.y, ll);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    if (whole) {
      const RowAt a = row_at(P, hk, r);
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      *reinterpret_cast<uint2*>(o_at(P, s, pc.b, a) + d) =
          make_uint2(ptx::pack_bf16(o.x * inv, o.y * inv), ptx::pack_bf16(o.z * inv, o.w * inv));
      if (d == 0 && P.lse != nullptr) P.lse[lse_at(P, s, pc.b, a)] = lse_of(mm, ll);
    } else {
      *reinterpret_cast<float4*>(P.part_o + (slot + row) * D + d) = o;
      if (d == 0) P.part_ml[slot + row] = make_float2(mm, ll);
    }
  }
  __syncthreads();   // before the next piece loads over the merge buffer
}

template <int D, bool FP8, int NT, int WM>
__global__ void __launch_bounds__(kThreads, 2) paged_stream_kernel(const __grid_constant__ StreamParams P) {
  using C = Cfg<D, FP8, NT, WM>;
  extern __shared__ __align__(128) uint8_t smem[];
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int total = total_units<C>(P);
  const int per = (total + gridDim.x - 1) / (int)gridDim.x;
  int x = min(total, (int)blockIdx.x * per);
  const int end = min(total, x + per);
  StreamMeta meta = {-1, 0, 0, 0};
  Walker<C> walk;
  while (x < end) {
    SeqRows s;
    const Piece pc = walk.at(P, x, end, s);
    if (pc.count <= 0) break;
    run_piece<C>(P, pc, s, smem);
    if (pc.first == 0 && pc.count < pc.tiles) meta = {pc.b, pc.seg, (x + pc.tiles - 1) / per, 0};
    x += pc.count;
  }
  if (P.split && threadIdx.x == 0) P.meta[blockIdx.x] = meta;
}

// Merges the parts of the segment that starts in CTA blockIdx.x and ends in a
// later one; one row per block, its warps sharing the parts.
template <int D, int RT>
__global__ void __launch_bounds__(kThreads) paged_merge_kernel(const __grid_constant__ StreamParams P) {
  constexpr int E = D / 32;   // columns per lane
  __shared__ float part[kThreads / 32][D];
  ptx::grid_dependency_wait();
  const StreamMeta me = P.meta[blockIdx.x];
  if (me.b < 0) return;
  const int hk = me.seg % P.c.heads_kv, rt = me.seg / P.c.heads_kv;
  const SeqRows s = load_seq(P.s, me.b, P.ws);
  const int row = blockIdx.y, r = rt * RT + row;
  if (r >= s.lq * P.group) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = me.last - (int)blockIdx.x + 1;
  // part 0 is slot 2c + 1 of the first CTA, the others slot 2c of theirs
  auto at = [&](int p) { return ((int64_t)2 * (blockIdx.x + p) + (p == 0 ? 1 : 0)) * RT + row; };
  float m = -INFINITY;
  for (int p = lane; p < n; p += 32) m = fmaxf(m, P.part_ml[at(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float l = 0.f;
  for (int p = lane; p < n; p += 32) {
    const float2 ml = P.part_ml[at(p)];
    l = fmaf(ptx::ex2(ml.x - base), ml.y, l);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kFull, l, o);
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 4
  for (int p = warp; p < n; p += kThreads / 32) {
    const float w = ptx::ex2(P.part_ml[at(p)].x - base);
    const float* v = P.part_o + at(p) * D + E * lane;
    if constexpr (E == 4) {
      const float4 x = __ldcs(reinterpret_cast<const float4*>(v));
      acc[0] = fmaf(w, x.x, acc[0]);
      acc[1] = fmaf(w, x.y, acc[1]);
      acc[2] = fmaf(w, x.z, acc[2]);
      acc[3] = fmaf(w, x.w, acc[3]);
    } else {
      const float2 x = __ldcs(reinterpret_cast<const float2*>(v));
      acc[0] = fmaf(w, x.x, acc[0]);
      acc[1] = fmaf(w, x.y, acc[1]);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) part[warp][E * lane + e] = acc[e];
  __syncthreads();
  const RowAt a = row_at(P, hk, r);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (threadIdx.x < D / 2) {
    const int d = 2 * threadIdx.x;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      x += part[w][d];
      y += part[w][d + 1];
    }
    *reinterpret_cast<uint32_t*>(o_at(P, s, me.b, a) + d) = ptx::pack_bf16(x * inv, y * inv);
  }
  if (threadIdx.x == 0 && P.lse != nullptr) P.lse[lse_at(P, s, me.b, a)] = lse_of(m, l);
}

template <int D, bool FP8, int NT, int WM>
cudaError_t launch_t(const StreamParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, FP8, NT, WM>;
  constexpr auto kern = paged_stream_kernel<D, FP8, NT, WM>;
  cudaError_t e = launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), kThreads, C::SMEM, stream); });
  if (e != cudaSuccess || !p.split) return e;
  const int64_t rows = (int64_t)p.s.seqlen_q * p.group;
  const unsigned ny = (unsigned)(rows < C::RT ? rows : C::RT);
  return launch_dependent(paged_merge_kernel<D, C::RT>, p, dim3((unsigned)grid, ny), kThreads, 0, stream);
}

template <int D, bool FP8>
cudaError_t launch_d(const StreamParams& p, int row_tile, int grid, cudaStream_t stream) {
  switch (row_tile) {
    case 8: return launch_t<D, FP8, 1, 1>(p, grid, stream);
    case 16: return launch_t<D, FP8, 2, 1>(p, grid, stream);
    case 32: return launch_t<D, FP8, 2, 2>(p, grid, stream);
    default: return launch_t<D, FP8, 2, 4>(p, grid, stream);
  }
}

}  // namespace

cudaError_t paged_stream_launch(const StreamParams& p, int head_dim, bool fp8, int row_tile, int grid,
                                cudaStream_t stream) {
  if (head_dim == 128)
    return fp8 ? launch_d<128, true>(p, row_tile, grid, stream) : launch_d<128, false>(p, row_tile, grid, stream);
  return fp8 ? launch_d<64, true>(p, row_tile, grid, stream) : launch_d<64, false>(p, row_tile, grid, stream);
}

}  // namespace af
