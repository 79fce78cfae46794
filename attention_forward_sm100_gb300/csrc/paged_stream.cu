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

template <int D_, bool FP8_, int WM_>
struct Cfg {
  static constexpr int D = D_, WM = WM_;
  static constexpr bool FP8 = FP8_;
  static constexpr int WK = 4 / WM;              // key groups
  static constexpr int KW = 16 * WM;             // keys of a group per tile
  static constexpr int RT = 16 * WM;             // rows of a row tile
  static_assert(WK * KW == kStreamTile, "the groups cover a tile");
  static constexpr int ROWB = FP8 ? D : 2 * D;   // bytes of a cached row
  static constexpr int CPR = ROWB / 16;          // 16-byte pieces of a row
  static constexpr int GT = 32 * WM;             // threads of a group
  static constexpr int RS = GT / CPR;            // rows a group loads at a time
  static constexpr int NL = KW / RS;             // loads per thread of K (and of V)
  static constexpr int KV = KW * ROWB;
  static constexpr int SC = FP8 ? KW * 4 : 0;
  static constexpr int STAGE = 2 * KV + 2 * SC;  // bytes of one group's stage
  static constexpr int STAGES = ROWB == 256 ? 3 : (ROWB == 128 ? 6 : 8);
  static constexpr int PITCH = D + 8;            // floats of a row in the group merge
  static constexpr int RING = WK * STAGES * STAGE;
  static constexpr int MERGE = WK * RT * (PITCH + 2) * 4;
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;   // the merge reuses the ring
  static_assert(SMEM <= 113 * 1024, "two CTAs per SM");
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
  u.tiles = P.split ? max(1, (u.r.lk + kStreamTile - 1) / kStreamTile) : 1;
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
  constexpr int D = C::D, WM = C::WM, KW = C::KW;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int wm = warp % WM, kg = warp / WM;
  const int gt = wm * 32 + lane;                  // thread within its key group
  const int hk = pc.seg % P.c.heads_kv, rt = pc.seg / P.c.heads_kv;
  const int rows = s.lq * P.group;
  const uint32_t ring = ptx::smem_u32(smem) + kg * (C::STAGES * C::STAGE);
  const int key_tiles = (s.lk + kStreamTile - 1) / kStreamTile;
  const int t0 = P.split ? pc.first : 0;
  const int n = P.split ? min(pc.count, key_tiles - t0) : key_tiles;

  // This thread's two rows: fragments of q and the keys each row sees.
  uint32_t qf[D / 16][4];
  int lim[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = rt * C::RT + 16 * wm + g + 8 * e;
    const bool ok = r < rows;
    const RowAt a = row_at(P, hk, ok ? r : 0);
    // (rows past the tile's end compute on zeros and are not stored)
    lim[e] = ok && P.causal ? min(s.lk, s.lk - s.lq + a.i + 1) : s.lk;
    const uint8_t* src = P.q + (P.s.cu_q != nullptr ? 0 : pc.b * P.q_b) + (int64_t)(s.q0 + a.i) * P.q_t + a.h * P.q_h;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      // depths of this lane's fragment: pairs at d and d + step
      const int d = C::FP8 ? 16 * (t + 4 * (kk >> 2)) + 4 * (kk & 3) : 16 * kk + 2 * t;
      const int step = C::FP8 ? 2 : 8;
      qf[kk][e] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 2 * d)) : 0u;
      qf[kk][2 + e] = ok ? __ldg(reinterpret_cast<const uint32_t*>(src + 2 * (d + step))) : 0u;
    }
  }
  // keys that every row of this warp sees need no mask
  int lim_min = min(lim[0], lim[1]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) lim_min = min(lim_min, __shfl_xor_sync(kFull, lim_min, o));

  const uint8_t* kbase = P.c.k + hk * P.c.k_head;
  const uint8_t* vbase = P.c.v + hk * P.c.v_head;
  const int page_mask = (1 << P.c.page_shift) - 1;
  const int lrow = gt / C::CPR, lcol = gt % C::CPR;

  // Pages of the 16-key blocks of a group's tile, fetched one tile ahead of
  // their use (the loads' addresses depend on them).
  int pages[WM];
  auto fetch_pages = [&](int j) {
    const int key0 = (t0 + j) * kStreamTile + kg * KW;
#pragma unroll
    for (int u = 0; u < WM; ++u)
      pages[u] = (j < n && key0 + 16 * u < s.lk) ? load_page(P.c, pc.b, (key0 + 16 * u) >> P.c.page_shift, P.ws) : 0;
  };
  auto load_tile = [&](int j) {
    const int key0 = (t0 + j) * kStreamTile + kg * KW;
    const uint32_t st = ring + (j % C::STAGES) * C::STAGE;
#pragma unroll
    for (int i = 0; i < C::NL; ++i) {
      const int row = lrow + i * C::RS;
      // rows of one load step lie in one 16-key block, or (RS = 32) in two
      const int page = C::RS <= 16 ? pages[(i * C::RS) >> 4]
                                   : (lrow < 16 ? pages[(i * C::RS) >> 4] : pages[((i * C::RS) >> 4) + (C::RS > 16)]);
      const bool ok = key0 + row < s.lk;
      const int64_t slot = (key0 + row) & page_mask;
      const uint8_t* ks = ok ? kbase + page * P.c.k_page + slot * P.c.k_tok + lcol * 16 : P.c.k;
      const uint8_t* vs = ok ? vbase + page * P.c.v_page + slot * P.c.v_tok + lcol * 16 : P.c.v;
      ptx::cp_async16(st + row * C::ROWB + C::swz_k(row, lcol) * 16, ks, ok);
      ptx::cp_async16(st + C::KV + row * C::ROWB + C::swz_v(row, lcol) * 16, vs, ok);
    }
    if constexpr (C::FP8) {
      // scales: 4 keys per 16 bytes; a piece that crosses the end is cut there
      if (gt < 2 * KW / 4) {
        const int which = gt / (KW / 4), k4 = 4 * (gt % (KW / 4));
        int page = pages[0];
#pragma unroll
        for (int u = 1; u < WM; ++u)
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

  float acc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

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
    const int key0 = (t0 + j) * kStreamTile + kg * KW;
    // ---- S = Q K^T
    float sc[KW / 8][4];
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) sc[i][e] = 0.f;
    if constexpr (!C::FP8) {
#pragma unroll
      for (int kk = 0; kk < D / 16; kk += 2)
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
          uint32_t b[4];
          const int row = 8 * i + (lane & 7);
          ptx::ldmatrix_x4(st + row * C::ROWB + C::swz_k(row, 2 * kk + (lane >> 3)) * 16, b);
          ptx::mma_16816(sc[i], qf[kk], b[0], b[1]);
          ptx::mma_16816(sc[i], qf[kk + 1], b[2], b[3]);
        }
    } else {
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int i = 0; i < KW / 8; ++i) {
          const int row = 8 * i + g;
          const uint4 w = ptx::ld_shared_v4(st + row * C::ROWB + C::swz_k(row, t + 4 * c) * 16);
          const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ptx::mma_16816(sc[i], qf[4 * c + e], ptx::e4m3x2_to_bf16x2(x[e] & 0xffffu), ptx::e4m3x2_to_bf16x2(x[e] >> 16));
        }
#pragma unroll
      for (int i = 0; i < KW / 8; ++i) {
        const uint2 k2 = ptx::ld_shared_v2(st + 2 * C::KV + (8 * i + 2 * t) * 4);
        const float k0 = __uint_as_float(k2.x), k1 = __uint_as_float(k2.y);
        sc[i][0] *= k0;
        sc[i][1] *= k1;
        sc[i][2] *= k0;
        sc[i][3] *= k1;
      }
    }
    // ---- mask, running maximum
    if (key0 + KW > lim_min) {
#pragma unroll
      for (int i = 0; i < KW / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (key0 + 8 * i + 2 * t + (e & 1) >= lim[e >> 1]) sc[i][e] = -INFINITY;
    }
    float mx[2] = {sc[0][0], sc[0][2]};
#pragma unroll
    for (int i = 0; i < KW / 8; ++i) {
      mx[0] = fmaxf(mx[0], fmaxf(sc[i][0], sc[i][1]));
      mx[1] = fmaxf(mx[1], fmaxf(sc[i][2], sc[i][3]));
    }
    bool grow = false;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFull, mx[e], 1));
      mx[e] = fmaxf(mx[e], __shfl_xor_sync(kFull, mx[e], 2)) * P.scale_log2;
      grow = grow || mx[e] > m[e] + 8.f;
    }
    if (__any_sync(kFull, grow)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (mx[e] > m[e] + 8.f) {
          const float alpha = ptx::ex2(m[e] - mx[e]);   // 0 at the first visible key
          m[e] = mx[e];
          l[e] *= alpha;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            acc[i][2 * e] *= alpha;
            acc[i][2 * e + 1] *= alpha;
          }
        }
      }
    }
    // ---- weights; a row that has seen no key yet keeps m = -inf and weights 0
    const float off[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
    for (int i = 0; i < KW / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[i][e] = ptx::ex2(fmaf(sc[i][e], P.scale_log2, -off[e >> 1]));
        l[e >> 1] += sc[i][e];
      }
    if constexpr (C::FP8) {
#pragma unroll
      for (int i = 0; i < KW / 8; ++i) {
        const uint2 v2 = ptx::ld_shared_v2(st + 2 * C::KV + C::SC + (8 * i + 2 * t) * 4);
        const float v0 = __uint_as_float(v2.x), v1 = __uint_as_float(v2.y);
        sc[i][0] *= v0;
        sc[i][1] *= v1;
        sc[i][2] *= v0;
        sc[i][3] *= v1;
      }
    }
    // ---- O += P V
#pragma unroll
    for (int kb = 0; kb < KW / 16; ++kb) {
      const uint32_t pf[4] = {
          ptx::pack_bf16(sc[2 * kb][0], sc[2 * kb][1]), ptx::pack_bf16(sc[2 * kb][2], sc[2 * kb][3]),
          ptx::pack_bf16(sc[2 * kb + 1][0], sc[2 * kb + 1][1]), ptx::pack_bf16(sc[2 * kb + 1][2], sc[2 * kb + 1][3])};
      if constexpr (!C::FP8) {
#pragma unroll
        for (int np = 0; np < D / 16; ++np) {
          uint32_t b[4];
          const int row = 16 * kb + (lane & 15);
          ptx::ldmatrix_x4_trans(st + C::KV + row * C::ROWB + C::swz_v(row, 2 * np + (lane >> 4)) * 16, b);
          ptx::mma_16816(acc[2 * np], pf, b[0], b[1]);
          ptx::mma_16816(acc[2 * np + 1], pf, b[2], b[3]);
        }
      } else {
        // lane (g, t): columns g * D/8 .. + D/8 of keys 2t, 2t+1, 2t+8, 2t+9
        uint32_t v[4][D / 32];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = 16 * kb + 2 * t + (e & 1) + 8 * (e >> 1);
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
          const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140), lo23 = __byte_perm(v[0][w], v[1][w], 0x7362);
          const uint32_t hi01 = __byte_perm(v[2][w], v[3][w], 0x5140), hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
          ptx::mma_16816(acc[4 * w], pf, ptx::e4m3x2_to_bf16x2(lo01 & 0xffffu), ptx::e4m3x2_to_bf16x2(hi01 & 0xffffu));
          ptx::mma_16816(acc[4 * w + 1], pf, ptx::e4m3x2_to_bf16x2(lo01 >> 16), ptx::e4m3x2_to_bf16x2(hi01 >> 16));
          ptx::mma_16816(acc[4 * w + 2], pf, ptx::e4m3x2_to_bf16x2(lo23 & 0xffffu), ptx::e4m3x2_to_bf16x2(hi23 & 0xffffu));
          ptx::mma_16816(acc[4 * w + 3], pf, ptx::e4m3x2_to_bf16x2(lo23 >> 16), ptx::e4m3x2_to_bf16x2(hi23 >> 16));
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(kFull, l[e], 1);
    l[e] += __shfl_xor_sync(kFull, l[e], 2);
  }
  ptx::cp_async_wait<0>();

  // ---- the key groups' results meet in shared memory (over the ring)
  float* buf = reinterpret_cast<float*>(smem);                          // [WK][RT][PITCH]
  float2* ml = reinterpret_cast<float2*>(buf + C::WK * C::RT * C::PITCH);   // [WK][RT]
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = 16 * wm + g + 8 * e;
    float* dst = buf + (kg * C::RT + r) * C::PITCH;
    if constexpr (!C::FP8) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
        *reinterpret_cast<float2*>(dst + 8 * i + 2 * t) = make_float2(acc[i][2 * e], acc[i][2 * e + 1]);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          *reinterpret_cast<float4*>(dst + (2 * t + c) * (D / 8) + 4 * i) =
              make_float4(acc[4 * i][2 * e + c], acc[4 * i + 1][2 * e + c], acc[4 * i + 2][2 * e + c],
                          acc[4 * i + 3][2 * e + c]);
    }
    if (t == 0) ml[kg * C::RT + r] = make_float2(m[e], l[e]);
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

template <int D, bool FP8, int WM>
__global__ void __launch_bounds__(kThreads, 2) paged_stream_kernel(const __grid_constant__ StreamParams P) {
  using C = Cfg<D, FP8, WM>;
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

template <int D, bool FP8, int WM>
cudaError_t launch_t(const StreamParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, FP8, WM>;
  constexpr auto kern = paged_stream_kernel<D, FP8, WM>;
  cudaError_t e = launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), kThreads, C::SMEM, stream); });
  if (e != cudaSuccess || !p.split) return e;
  const int64_t rows = (int64_t)p.s.seqlen_q * p.group;
  const unsigned ny = (unsigned)(rows < C::RT ? rows : C::RT);
  return launch_dependent(paged_merge_kernel<D, C::RT>, p, dim3((unsigned)grid, ny), kThreads, 0, stream);
}

template <int D, bool FP8>
cudaError_t launch_d(const StreamParams& p, int row_groups, int grid, cudaStream_t stream) {
  switch (row_groups) {
    case 1: return launch_t<D, FP8, 1>(p, grid, stream);
    case 2: return launch_t<D, FP8, 2>(p, grid, stream);
    default: return launch_t<D, FP8, 4>(p, grid, stream);
  }
}

}  // namespace

cudaError_t paged_stream_launch(const StreamParams& p, int head_dim, bool fp8, int row_groups, int grid,
                                cudaStream_t stream) {
  if (head_dim == 128)
    return fp8 ? launch_d<128, true>(p, row_groups, grid, stream) : launch_d<128, false>(p, row_groups, grid, stream);
  return fp8 ? launch_d<64, true>(p, row_groups, grid, stream) : launch_d<64, false>(p, row_groups, grid, stream);
}

}  // namespace af
