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
#include "paged_walk.cuh"

namespace af {
namespace {

constexpr int kThreads = 128;

// NT * 8 rows per warp, WM warps to a key group.
template <int D_, bool FP8_, int NT_, int WM_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WM = WM_;
  static constexpr bool FP8 = FP8_;
  static constexpr int CTAS = stream_ctas(FP8 ? D : 2 * D, 8 * NT * WM);
  static constexpr int WK = 4 / WM;              // key groups
  static constexpr int RT = 8 * NT * WM;         // rows of a row tile
  static constexpr int ROWB = FP8 ? D : 2 * D;   // bytes of a cached row
  static constexpr int KW = stream_tile(ROWB, WM) / WK;   // keys of a group per tile
  static constexpr int TILE = KW * WK;
  static constexpr int BLOCKS = KW / 16;         // 16-key blocks of a group's tile
  static constexpr int CPR = ROWB / 16;          // 16-byte pieces of a row
  static constexpr int GT = 32 * WM;             // threads of a group
  static constexpr int RS = GT / CPR;            // rows a group loads at a time
  static_assert(RS <= 16, "the rows of a load lie in one 16-key block");
  static constexpr int NL = KW / RS;             // loads per thread of K (and of V)
  static constexpr int KV = KW * ROWB;
  static constexpr int SC = FP8 ? KW * 4 : 0;
  static constexpr int STAGE = 2 * KV + 2 * SC;  // bytes of one group's stage
  // At the end of a segment a group leaves its part of O in the stage that it
  // has just used up, or, where that is too small, in room of its own.
  static constexpr int PART = RT * D * 4;
  static constexpr bool OWN_PART = PART > STAGE;
  static constexpr int STAGES = min_int(8, (196608 / CTAS - (OWN_PART ? WK * PART : 0)) / (WK * 2 * KV));
  static constexpr int RING = WK * STAGES * STAGE;
  static constexpr int OFF_ML = RING + (OWN_PART ? WK * PART : 0);   // [WK][RT] (maximum, sum)
  static constexpr int SMEM = OFF_ML + WK * RT * 8;
  static constexpr int FT = kThreads;   // all threads finish a piece
  __device__ static int ftid() { return threadIdx.x; }
  __device__ static void fsync() { __syncthreads(); }
  // Byte offset of group k's part, `last` being its stage's in the group's ring.
  __device__ static int part_at(int k, int last) { return OWN_PART ? RING + k * PART : k * (STAGES * STAGE) + last; }
  static_assert(STAGES >= 3 && SMEM <= 226 * 1024 / CTAS, "the CTAs per SM");
  // Depths of a lane's q pair kk: this one and the next, and those Q_STEP behind.
  static constexpr int Q_STEP = FP8 ? 2 : 8;
  __device__ static int q_depth(int kk, int t) { return FP8 ? 16 * (t + 4 * (kk >> 2)) + 4 * (kk & 3) : 16 * kk + 2 * t; }
  // Column of depth d of row r there: rows 2 t and 2 t + 1 shifted by 8 t banks.
  __device__ static int part_col(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }
  // Position of 16-byte piece `c` of row `r` in a stage (bank conflicts).
  __device__ static int swz_k(int r, int c) {
    return FP8 ? (CPR == 8 ? c ^ ((r & 1) << 2) : c) : c ^ (r & 7);
  }
  __device__ static int swz_v(int r, int c) { return FP8 && CPR == 4 ? c ^ ((r >> 1) & 3) : c ^ (r & 7); }
};

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
    if constexpr (C::FP8) {
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
  // e4m3: the accumulator is in units of vref / 2^7, vref a power of two at
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
    if constexpr (!C::FP8) {
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
          vs[i][e] = scale_sm[KW + 16 * i + g + 8 * e];
          top = fmaxf(top, fabsf(vs[i][e]));
          // (keys behind the end have scale 0 and weight 0)
          if (key0 + 16 * i + g + 8 * e < s.lk) low = fminf(low, fabsf(vs[i][e]));
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
        // (key, key) pairs of each depth
        auto product = [&](auto f16) {
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

  if constexpr (C::FP8) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][x][e] *= vref * 0.0078125f;
  }

  if (first + pc.count < end) {
    next = walk.at(P, first + pc.count, end, next_rows);
    load_q<C>(P, next, next_rows, wm, qf);
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
          if constexpr (C::FP8) {
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
  auto part_of = [&](int k) { return n > 0 ? reinterpret_cast<const float*>(smem + C::part_at(k, last)) : nullptr; };
  finish_piece<C>(P, pc, s, ml, part_of, first, per);
}

template <int D, bool FP8, int NT, int WM>
__global__ void __launch_bounds__(kThreads, (Cfg<D, FP8, NT, WM>::CTAS))
    paged_stream_kernel(const __grid_constant__ StreamParams P) {
  using C = Cfg<D, FP8, NT, WM>;
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
  load_q<C>(P, pc, s, (int)(threadIdx.x >> 5) % C::WM, qf);
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

template <int D, bool FP8, int NT, int WM>
cudaError_t launch_t(const StreamParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, FP8, NT, WM>;
  constexpr auto kern = paged_stream_kernel<D, FP8, NT, WM>;
  return launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), kThreads, C::SMEM, stream); });
}

template <int D, bool FP8>
cudaError_t launch_d(const StreamParams& p, int row_tile, int grid, cudaStream_t stream) {
  switch (row_tile) {
    case 8: return launch_t<D, FP8, 1, 1>(p, grid, stream);
    case 16: return launch_t<D, FP8, 2, 1>(p, grid, stream);
    default: return launch_t<D, FP8, 2, 2>(p, grid, stream);
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
