// Attention of a few new tokens over a paged cache of e2m1 codes.
//
// The work, its division among CTAs and the joining of parts are those of
// paged_stream.cu (paged_walk.cuh). What differs is that 4-bit keys are so few
// bytes that the instructions of loading and converting them bound the kernel, not
// HBM: 16 keys of one head of 128 depths are 2432 bytes, 103 cycles of an SM at the
// copy rate, and about 250 warp instructions at best. So
//   * one CTA per SM whose warps have roles, so that those that compute do nothing else.
//     Two load, one the keys and one the values. (With each computing thread copying its
//     own 16-byte pieces 413 instructions went into 16 keys, and 16 sequences of up to
//     32768 keys, GQA 32/8, took 96 us; one warp that issues TMA boxes and bulk copies,
//     six for 32 keys, takes 60 ns for each: 184 us.) One brings the next piece's q into
//     shared memory as the instructions want it. One reduces what the others leave of a
//     piece, and joins the parts of cut segments.
//   * twelve warps (eight for more than eight rows) compute. Warp w takes 32 keys at a
//     time, the CTA's w-th, (w + 12)-th, ..., from a ring of its own, whatever piece they
//     belong to. With three CTAs per SM of four computing warps each, which stopped to
//     finish every piece, the last CTA ended when the first had been idle for 20 of 84 us.
//   * codes become f16 two at a time and are multiplied by their block's scale,
//     which is exact (two significant bits times four). S^T = K Q^T and O^T = V^T P^T
//     as in paged_stream.cu; the vectors' scales are applied to the fp32 scores and
//     weights. For V^T, whose operands are pairs of keys, two keys' bytes are merged
//     into (key, key) pairs of a depth before they are converted.
// Slots at or past the sequence's end are not read (their shared memory is
// zeroed), so whatever they hold cannot reach a result.
//
// Every wait is bounded: when one runs out, the error is recorded, nothing waits any
// more, and the CTA runs to its end on whatever is in shared memory.
#include <cuda_fp16.h>
#include <math.h>

#include <type_traits>

#include "launch.cuh"
#include "paged_walk.cuh"

namespace af {
namespace {

template <int D_, int NT_, int WM_>
struct Cfg {
  static constexpr int D = D_, NT = NT_, WM = WM_;
  static constexpr int RT = 8 * NT * WM;
  static constexpr int W = NT == 1 ? 12 : 8, WK = W / WM;   // computing warps, key groups of them
  static constexpr int LOADER = W, FEEDER = W + 2, FINISHER = W + 3, THREADS = 32 * (W + 4);
  static constexpr int KW = 32, NB = KW / 16;       // keys of a step of a group, 16-key blocks of them
  static constexpr int TILE = stream4_tile, STEPS = TILE / KW;   // keys of a unit of work, steps of it
  static constexpr int ROWB = D / 2, BK = D / 16;   // bytes of a row's codes, block scales of it
  static constexpr int VB = D / 64;                 // 4-byte words of codes that a lane holds of a key of V
  // A stage, one step's: codes of K and V, and in another place block scales of both,
  // scales of both.
  static constexpr int AT_V = KW * ROWB, CODES = 2 * AT_V;
  static constexpr int AT_VB = KW * BK, AT_KS = 2 * AT_VB, AT_VS = AT_KS + 4 * KW, SCALES = AT_VS + 4 * KW;
  static constexpr int PART = RT * D * 4;           // a group's part of O
  static constexpr int JOBS = 4;                    // pieces that the loading warp is ahead at most
  static constexpr int QF = WM * NT * (D / 16) * 256, Q = QF + 4 * RT;   // q of a piece, and its rows' factors
  static constexpr int REST = WK * PART + WK * RT * 8 + 2 * Q + JOBS * 48 + JOBS * 32;
  static constexpr int PER = min_int(6, (232448 - 1024 - REST) / (WK * (CODES + SCALES + 16)));   // stages of a group
  static constexpr int S = PER * WK;
  static_assert(PER >= 3, "loads in flight");
  static constexpr int AT_SC = S * CODES, AT_PART = AT_SC + S * SCALES, AT_ML = AT_PART + WK * PART, AT_Q = AT_ML + WK * RT * 8, AT_JOB = AT_Q + 2 * Q,
                       AT_BAR = AT_JOB + JOBS * 48, SMEM = AT_BAR + 16 * S + JOBS * 32;
  static_assert(AT_PART % 16 == 0 && AT_Q % 16 == 0 && AT_JOB % 16 == 0 && AT_BAR % 8 == 0, "vector accesses");
  __device__ static int part_col(int r, int d) { return d ^ (((r >> 1) & 3) << 3); }
  // lane t's depths of a key: D / 4 from t D / 4 on, four for each q pair
  static constexpr int Q_STEP = 2;
  __device__ static int q_depth(int kk, int t) { return D / 4 * t + 4 * kk; }
  // Where 16-byte piece `c` of row `r` is (bank conflicts).
  __device__ static int swz(int r, int c) { return D == 128 ? c ^ ((r >> 1) & 3) : c ^ ((r >> 2) & 1); }
  // Which row of an 8-key group is key m of the instructions (any order will do, as
  // long as K and V agree): this one spreads the rows that lanes read together, 2 t of
  // V and two (D = 64: four) neighbours of K, over all banks.
  __device__ static int key_row(int m) { return D == 128 ? m ^ ((m >> 1) & 1) : m ^ ((m >> 2) & 1); }
  // the warp that finishes
  static constexpr int FT = 32;
  __device__ static int ftid() { return threadIdx.x & 31; }
  __device__ static void fsync() { __syncwarp(); }
};

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }
__device__ __forceinline__ uint32_t as_bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

// Barriers (8 bytes each) and what is shared through them.
struct Pipe {
  uint32_t full, empty;     // of stage 0: a step's keys are there, its group is done with them
  // of job 0: the piece is described; its q is there; every warp has left its part; that
  // has been used, and nothing of the piece is needed any more
  uint32_t named, ready, left, done;
  int* jobs;                // 12 words each
  volatile int* over;       // a wait has run out
  uint32_t* ws;

  // Whether a wait of some warp has run out, for all lanes alike.
  __device__ __forceinline__ bool given_up() const { return __any_sync(kFull, *over); }
  // Whether the barrier's phase has ended (else a wait has run out).
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, int role) const {
    return ptx::mbar_try_wait(bar, parity) || wait_long(bar, parity, role);
  }
  __device__ __forceinline__ bool wait_long(uint32_t bar, uint32_t parity, int role) const {
    uint64_t since = 0;
    for (uint32_t i = 1;; ++i) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if ((i & 15u) == 0u) {
        if (*over) return false;
        const uint64_t now = ptx::globaltimer();
        if (since == 0) since = now;
        if (now - since > 2000000000ull) {
          if (atomicCAS(&ws[kWsErrorCode], 0u, (uint32_t)kDevErrTimeout) == 0u)
            atomicExch(&ws[kWsErrorInfo], (blockIdx.x << 16) | ((uint32_t)role << 8));
          *over = 1;
          return false;
        }
      }
    }
  }
};

// A piece, its sequence's rows, its first unit among all and its first step among the
// CTA's, as the loading warp hands them to the others; count 0: there are no more.
struct Job {
  Piece pc;
  SeqRows s;
  int first, step;
};
template <class C>
__device__ __forceinline__ uint32_t slot_of(int k) { return k % C::JOBS; }
template <class C>
__device__ __forceinline__ uint32_t phase_of(int k) { return (uint32_t)(k / C::JOBS) & 1u; }
template <class C>
__device__ __forceinline__ void hand_over(const Pipe& pipe, int k, const Job& j) {
  pipe.wait(pipe.done + 8 * slot_of<C>(k), phase_of<C>(k) ^ 1u, 2);
  if ((threadIdx.x & 31) == 0) {
    int4* to = reinterpret_cast<int4*>(pipe.jobs + 12 * slot_of<C>(k));
    to[0] = make_int4(j.pc.b, j.pc.seg, j.pc.first, j.pc.count);
    to[1] = make_int4(j.pc.tiles, j.s.lq, j.s.lk, j.s.q0);
    to[2] = make_int4(j.first, j.step, 0, 0);
    ptx::mbar_arrive(pipe.named + 8 * slot_of<C>(k));
  }
  __syncwarp();
}
template <class C>
__device__ __forceinline__ Job job_at(const Pipe& pipe, int k) {
  const int4* from = reinterpret_cast<const int4*>(pipe.jobs + 12 * slot_of<C>(k));
  const int4 a = from[0], b = from[1], c = from[2];
  return {{a.x, a.y, a.z, a.w, b.x}, {b.y, b.z, b.w}, c.x, c.y};
}
// First key and steps of a piece.
template <class C>
__device__ __forceinline__ void piece_steps(const StreamParams& P, const Piece& pc, const SeqRows& s, int& key, int& steps) {
  int t0, n;
  piece_tiles<C>(P, pc, s, t0, n);
  key = t0 * C::TILE;
  steps = n > 0 ? (min(n * C::TILE, s.lk - key) + C::KW - 1) / C::KW : 0;
}

// The warps that load, `v` false the keys, true the values: every step of this CTA's
// pieces, in order, eight steps (a turn) at a time. A warp that loads is bound by its
// own instructions' latencies, so little is done per step: a lane has two of a turn's
// sixteen 16-key blocks for itself and copies one 16-byte piece of each of their rows (D
// = 64: of eight rows); where blocks lie is worked out for 32 at once; and barriers, whose
// instructions take a warp 60 cycles and 250 if all lanes use them, are met by one lane
// for each step. Cycles for a step, in the order of these changes: 480, 317, 150.
template <class C>
__device__ __forceinline__ void load_steps(const StreamParams& P, Walker<C> walk, const Pipe& pipe, uint32_t smem, int x,
                                           int end, bool v) {
  constexpr int CPR = C::ROWB / 16, ROWS = 4 * CPR;       // 16-byte pieces of a row; rows that a lane copies of
  constexpr int BPL = C::BK / 4;                          // 16-byte pieces of a block's block scales, a lane's
  static_assert(CPR == 4 || CPR == 2, "four lanes to a block");
  const int lane = threadIdx.x & 31;
  const int page_mask = (1 << P.c.page_shift) - 1;
  const int blk = lane >> 2, quarter = lane & 3;          // first block of a turn's two, which of its lanes
  const int row = CPR == 4 ? 0 : 8 * (quarter >> 1), col = quarter % CPR;   // this lane's first row, piece of each
  const int64_t page_bytes = v ? P.c.v_page : P.c.k_page, tok_bytes = v ? P.c.v_tok : P.c.k_tok;
  const int64_t mine = row * tok_bytes + col * 16;
  const uint8_t* const codes = v ? P.c.v : P.c.k;
  const uint8_t* const blocks = (v ? P.blocks.v : P.blocks.k) + quarter * 16;
  const float* const scales = (v ? P.c.v_scale : P.c.k_scale) + quarter * 4;
  // places in a stage
  const uint32_t in_codes = smem + (v ? C::AT_V : 0) + (16 * (blk & 1) + row) * C::ROWB;
  const uint32_t in_blocks = smem + C::AT_SC + (v ? C::AT_VB : 0) + 16 * (blk & 1) * C::BK + quarter * 16;
  const uint32_t in_scales = smem + C::AT_SC + (v ? C::AT_VS : C::AT_KS) + 16 * (blk & 1) * 4 + quarter * 16;
  auto around = [](uint32_t st) { return st >= (uint32_t)C::S ? st - C::S : st; };
  int step = 0, k = 0;
  uint32_t stage = 0, parity = 1;   // of the next step
  // Steps are announced once their copies are there, LAG turns later.
  constexpr int LAG = C::S >= 32 ? 2 : 1;
  static_assert(C::S >= 8 * (LAG + 2), "whoever a turn waits for has been told of its steps");
  uint32_t told = 0;                // the stage that is announced next
  int turns = 0;
  uint32_t sizes = 0;               // turns in flight; their steps, four bits each, the oldest lowest
  auto announce = [&]() {
    const uint32_t n = sizes & 15u;
    sizes >>= 4;
    __syncwarp();
    if ((uint32_t)lane < n) ptx::mbar_arrive(pipe.full + 8 * around(told + lane));
    told = around(told + n);
  };
  auto flush = [&]() {
    ptx::cp_async_wait_all();
    while (sizes != 0u) announce();
    turns = 0;
  };
  bool fine = !pipe.given_up();
  while (x < end && fine) {
    SeqRows s;
    const Piece pc = walk.at(P, x, end, s);
    if (!v) {
      // (whoever has to be done with piece k - 4 may be waiting for what is not announced yet)
      if (sizes != 0u && !ptx::mbar_test_wait(pipe.done + 8 * slot_of<C>(k), phase_of<C>(k) ^ 1u)) flush();
      hand_over<C>(pipe, k, {pc, s, x, step});
    }
    ++k;
    x += max(1, pc.count);
    int key, n;
    piece_steps<C>(P, pc, s, key, n);
    step += n;
    const int hk = head_of(P, pc.seg);
    const int32_t* const table = P.c.table + (int64_t)pc.b * P.c.table_stride;
    const uint8_t* const head = codes + hk * (v ? P.c.v_head : P.c.k_head);
    // 32 blocks, two turns, one a lane: where their codes are, and keys in front of their
    // scales. The next 32 pages' numbers are on their way.
    auto page_from = [&](int first) {
      const int at = first + 16 * lane;
      return at < s.lk ? __ldg(table + (at >> P.c.page_shift)) : 0;
    };
    uint64_t code_at = 0;
    int64_t scale_at = 0;
    int next = n > 0 ? page_from(key) : 0;
#pragma unroll 1
    for (int j = 0; j < n; j += 8, key += 256) {
      if ((j & 15) == 0) {
        const int at = key + 16 * lane, slot = at & page_mask;
        const int page = at < s.lk ? checked_page(P.c, next, pc.b, P.ws) : 0;
        code_at = reinterpret_cast<uint64_t>(head + page * page_bytes + slot * tok_bytes);
        scale_at = (((int64_t)page * P.c.heads_kv + hk) << P.c.page_shift) + slot;
        next = page_from(key + 512);
      }
      const int m = min(8, n - j);
      if (lane < m) {
        const uint32_t st = around(stage + lane);
        fine = pipe.wait(pipe.empty + 8 * st, parity ^ (st < stage ? 1u : 0u), 1);
      }
      fine = __all_sync(kFull, fine);
      if (!fine) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int from_lane = 2 * (j & 15) + 8 * h + blk;
        const uint8_t* from = reinterpret_cast<const uint8_t*>(__shfl_sync(kFull, code_at, from_lane)) + mine;
        const int64_t at = __shfl_sync(kFull, scale_at, from_lane);
        if (4 * h + (blk >> 1) < m) {
          const int left = s.lk - (key + 16 * (8 * h + blk));   // keys from the block's first on
          const uint32_t st = around(stage + 4 * h + (blk >> 1));
          const uint32_t to = in_codes + st * C::CODES, to_sc = st * C::SCALES;
          if (left >= 16) {
#pragma unroll
            for (int y = 0; y < ROWS; ++y) {
              ptx::cp_async16(to + y * C::ROWB + C::swz(y, col) * 16, from);
              from += tok_bytes;
            }
#pragma unroll
            for (int i = 0; i < BPL; ++i) ptx::cp_async16(to_sc + in_blocks + 64 * i, blocks + at * C::BK + 64 * i);
            ptx::cp_async16(to_sc + in_scales, scales + at);
          } else {   // slots at or behind the end are zeros
#pragma unroll 1
            for (int y = 0; y < ROWS; ++y) {
              ptx::cp_async16(to + y * C::ROWB + C::swz(y, col) * 16, left > row + y ? from : codes, left > row + y);
              from += tok_bytes;
            }
#pragma unroll
            for (int i = 0; i < BPL; ++i) {
              const int bytes = min(16, max(0, left * C::BK - quarter * 16 - 64 * i));
              ptx::cp_async16_part(to_sc + in_blocks + 64 * i, bytes ? blocks + at * C::BK + 64 * i : blocks, bytes);
            }
            const int bytes = min(16, max(0, (left - quarter * 4) * 4));
            ptx::cp_async16_part(to_sc + in_scales, bytes ? scales + at : scales, bytes);
          }
        }
        __syncwarp();
      }
      const uint32_t before = stage;
      stage = around(stage + m);
      if (stage < before) parity ^= 1u;
      ptx::cp_async_commit();
      sizes |= (uint32_t)m << (4 * turns);
      if (turns < LAG) {
        ++turns;
      } else {
        ptx::cp_async_wait<LAG>();
        announce();
      }
    }
  }
  flush();   // (and nothing is left in flight when the CTA ends)
  if (!v) hand_over<C>(pipe, k, {{0, 0, 0, 0, 1}, {0, 0, 0}, 0, 0});
}

// The warp that feeds q: of every piece, as f16 in the order of the instructions, times
// the power of two that brings a row's largest magnitude to [2^14, 2^15), which is exact
// down to 2^-38 of that, and the factors that undo it.
template <class C>
__device__ __forceinline__ void feed_q(const StreamParams& P, uint8_t* smem, const Pipe& pipe) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll 1
  for (int k = 0;; ++k) {
    pipe.wait(pipe.named + 8 * slot_of<C>(k), phase_of<C>(k), 3);
    const Job job = job_at<C>(pipe, k);
    if (job.pc.count == 0 || pipe.given_up()) return;
    // (its place is piece k - 2's, which everyone has read)
    if (k >= 2) pipe.wait(pipe.left + 8 * slot_of<C>(k - 2), phase_of<C>(k - 2), 3);
    uint8_t* const to = smem + C::AT_Q + (k & 1) * C::Q;
#pragma unroll 1
    for (int wm = 0; wm < C::WM; ++wm) {
      uint32_t qf[C::NT][C::D / 16][2];
      load_q<C>(P, job.pc, job.s, wm, qf);
#pragma unroll
      for (int x = 0; x < C::NT; ++x) {
        uint32_t top = 0u;
#pragma unroll
        for (int kk = 0; kk < C::D / 16; ++kk)
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
        for (int kk = 0; kk < C::D / 16; ++kk) {
          uint32_t h[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint32_t w = qf[x][kk][c];
            h[c] = ptx::pack_f16(__uint_as_float(w << 16) * up, __uint_as_float(w & 0xffff0000u) * up);
          }
          *reinterpret_cast<uint2*>(to + ((wm * C::NT + x) * (C::D / 16) + kk) * 256 + lane * 8) = make_uint2(h[0], h[1]);
        }
        if (t == 0)
          reinterpret_cast<float*>(to + C::QF)[8 * (wm * C::NT + x) + g] =
              __uint_as_float((uint32_t)max(e - 14, 1) << 23) * P.scale_log2;
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(pipe.ready + 8 * slot_of<C>(k));
  }
}

// The warp that finishes: every piece once all have left their parts.
template <class C>
__device__ __forceinline__ void finish_pieces(const StreamParams& P, uint8_t* smem, const Pipe& pipe, int per) {
#pragma unroll 1
  for (int k = 0;; ++k) {
    pipe.wait(pipe.named + 8 * slot_of<C>(k), phase_of<C>(k), 4);
    const Job job = job_at<C>(pipe, k);
    if (job.pc.count == 0) return;
    pipe.wait(pipe.left + 8 * slot_of<C>(k), phase_of<C>(k), 4);
    if (pipe.given_up()) return;
    int key, steps;
    piece_steps<C>(P, job.pc, job.s, key, steps);
    auto part = [&](int i) -> const float* {   // group i's steps are those of its number modulo WK
      int behind = (i - job.step) % C::WK;
      if (behind < 0) behind += C::WK;
      return behind < steps ? reinterpret_cast<const float*>(smem + C::AT_PART + i * C::PART) : nullptr;
    };
    finish_piece<C>(P, job.pc, job.s, reinterpret_cast<const float2*>(smem + C::AT_ML), part, job.first, per);
    C::fsync();
    if (C::ftid() == 0) ptx::mbar_arrive(pipe.done + 8 * slot_of<C>(k));
  }
}

// A computing warp's share of every piece.
template <class C>
__device__ __forceinline__ void compute(const StreamParams& P, uint8_t* smem, const Pipe& pipe) {
  constexpr int D = C::D, WM = C::WM, NT = C::NT, KW = C::KW, NB = C::NB;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3, gk = C::key_row(g);
  const int wm = warp % WM, kg = warp / WM;
  // This lane's places in a stage (added to constants, the swizzle depending on the
  // row among eight alone): its key of K, the words of two keys of V, their scales.
  const uint32_t smem0 = ptx::smem_u32(smem);
  const uint32_t at_k = gk * C::ROWB + (D == 128 ? C::swz(gk, t) * 16 : C::swz(gk, t >> 1) * 16 + (t & 1) * 8);
  const uint32_t at_kb = gk * C::BK + (D == 128 ? 2 * t : t);   // (of the scales' place, as those that follow)
  const uint32_t at_sc = C::AT_KS + gk * 4;
  uint32_t at_v[2], at_vb[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = C::key_row(2 * t + e);
    at_v[e] = C::AT_V + r * C::ROWB + (D == 128 ? C::swz(r, g >> 1) * 16 + (g & 1) * 8 : C::swz(r, g >> 2) * 16 + (g & 3) * 4);
    at_vb[e] = C::AT_VB + r * C::BK + (D == 128 ? g : g >> 1);
  }
  int at = kg;   // the next step of this group, among the CTA's
  int turn = 0;  // of its stages
  uint32_t parity = 0;

#pragma unroll 1
  for (int k = 0;; ++k) {
  pipe.wait(pipe.named + 8 * slot_of<C>(k), phase_of<C>(k), 5);
  int key0, n, lim_min;
  // Rows row0 + 8 x + 2 t and + 1 are this lane's columns of the score and output
  // tiles: the keys they see, and the factor of their scaled q.
  int lim[NT][2];
  {
    const Job job = job_at<C>(pipe, k);
    if (job.pc.count == 0 || pipe.given_up()) return;
    const int rows = job.s.lq * P.group, row0 = row_tile_of(P, job.pc.seg) * C::RT + 8 * NT * wm;
    piece_steps<C>(P, job.pc, job.s, key0, n);
    key0 += (at - job.step) * KW;
    n += job.step;
    const int lk = job.s.lk;
    lim_min = lk;
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
  pipe.wait(pipe.ready + 8 * slot_of<C>(k), phase_of<C>(k), 5);
  const uint32_t at_q = smem0 + C::AT_Q + (k & 1) * C::Q + wm * NT * (D / 16) * 256 + lane * 8;
  float qscale[NT][2];
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
      qscale[x][e] = ptx::ld_shared_f32(smem0 + C::AT_Q + (k & 1) * C::Q + C::QF + 4 * (8 * (wm * NT + x) + 2 * t + e));

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
  const bool some = at < n;

#pragma unroll 1
  for (; at < n; at += C::WK, key0 += C::WK * KW) {
    const int stage = turn * C::WK + kg;
    const uint32_t st = smem0 + stage * C::CODES, ss = smem0 + C::AT_SC + stage * C::SCALES;
    pipe.wait(pipe.full + 8 * stage, parity, 0);
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
          s2[i][e] = as_half2(ptx::e4m3x2_to_f16x2(ptx::ld_shared_u16(ss + at_kb + row * C::BK)));
        } else {
          const uint2 v = ptx::ld_shared_v2(st + at_k + row * C::ROWB);
          w[i][e][0] = v.x; w[i][e][1] = v.y;
          s2[i][e] = as_half2(ptx::e4m3x2_to_f16x2(ptx::ld_shared_u8(ss + at_kb + row * C::BK)));
        }
      }
    }
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      uint2 qw[NT][2];
#pragma unroll
      for (int x = 0; x < NT; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) qw[x][y] = ptx::ld_shared_v2(at_q + (x * (D / 16) + 2 * c + y) * 256);
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
      const float k0 = ptx::ld_shared_f32(ss + at_sc + 64 * i), k1 = ptx::ld_shared_f32(ss + at_sc + 64 * i + 32);
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
        vk[i][e] = ptx::ld_shared_f32(ss + at_sc + 4 * KW + 64 * i + 32 * e);
        top = fmaxf(top, fabsf(vk[i][e]));
        low = fminf(low, fabsf(vk[i][e]));   // (0 behind the end: bf16 will do for a last tile)
      }
    const bool plain = __all_sync(kFull, top <= vref && low >= vref * 0.0625f);
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
          b[e] = ptx::ld_shared_u8(ss + at_vb[e & 1] + row * C::BK);
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
    if (++turn == C::PER) {
      turn = 0;
      parity ^= 1u;
    }
  }
#pragma unroll
  for (int x = 0; x < NT; ++x)
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[x][e] += __shfl_xor_sync(kFull, l[x][e], o);

  // ---- What this warp has of the piece, for those that finish it; the place was piece
  // k - 1's.
  if (k > 0) pipe.wait(pipe.done + 8 * slot_of<C>(k - 1), phase_of<C>(k - 1), 5);
  float2* ml = reinterpret_cast<float2*>(smem + C::AT_ML);   // [WK][RT]
  if (some) {
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
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(pipe.left + 8 * slot_of<C>(k));
  }
}

template <int D, int NT, int WM>
__global__ void __launch_bounds__((Cfg<D, NT, WM>::THREADS), 1)
    paged_stream4_kernel(const __grid_constant__ StreamParams P) {
  using C = Cfg<D, NT, WM>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int over;
  Pipe pipe;
  pipe.full = ptx::smem_u32(smem) + C::AT_BAR;
  pipe.empty = pipe.full + 8 * C::S;
  pipe.named = pipe.empty + 8 * C::S;
  pipe.ready = pipe.named + 8 * C::JOBS;
  pipe.left = pipe.ready + 8 * C::JOBS;
  pipe.done = pipe.left + 8 * C::JOBS;
  pipe.jobs = reinterpret_cast<int*>(smem + C::AT_JOB);
  pipe.over = &over;
  pipe.ws = P.ws;
  for (int i = threadIdx.x; i < C::S; i += C::THREADS) {
    ptx::mbar_init(pipe.full + 8 * i, 2);   // (the warps that load)
    ptx::mbar_init(pipe.empty + 8 * i, C::WM);
  }
  if (threadIdx.x < C::JOBS) {
    ptx::mbar_init(pipe.named + 8 * threadIdx.x, 1);
    ptx::mbar_init(pipe.ready + 8 * threadIdx.x, 1);
    ptx::mbar_init(pipe.left + 8 * threadIdx.x, C::W);
    ptx::mbar_init(pipe.done + 8 * threadIdx.x, 1);
  }
  if (threadIdx.x == 0) over = 0;
  ptx::fence_mbar_init();
  __syncthreads();
  ptx::grid_dependency_wait();
  ptx::launch_dependents();
  const int warp = threadIdx.x >> 5;
  if (warp < C::W) {
    compute<C>(P, smem, pipe);
    return;
  }
  if (warp == C::FEEDER) {
    feed_q<C>(P, smem, pipe);
    return;
  }
  // The units of a CTA are needed to load and to finish.
  Walker<C> walk;
  const int total = walk.start(P);
  const int teams = (int)gridDim.x / P.team;
  const int per = (total + teams - 1) / teams;
  const int x = min(total, (int)blockIdx.x / P.team * per), end = min(total, x + per);
  if (warp == C::FINISHER) {
    finish_pieces<C>(P, smem, pipe, per);
  } else {
    if (P.s.batch > 32 && x < end) walk.seek(P, x);
    load_steps<C>(P, walk, pipe, ptx::smem_u32(smem), x, end, warp != C::LOADER);
  }
}

template <int D, int NT, int WM>
cudaError_t launch_t(const StreamParams& p, int grid, cudaStream_t stream) {
  using C = Cfg<D, NT, WM>;
  constexpr auto kern = paged_stream4_kernel<D, NT, WM>;
  return launch_with_smem<kern>(
      C::SMEM, [&]() { return launch_dependent(kern, p, dim3((unsigned)grid), C::THREADS, C::SMEM, stream); });
}

template <int D>
cudaError_t launch_d(const StreamParams& p, int row_tile, int grid, cudaStream_t stream) {
  switch (row_tile) {
    case 8: return launch_t<D, 1, 1>(p, grid, stream);
    case 16: return launch_t<D, 2, 1>(p, grid, stream);
    default: return launch_t<D, 2, 2>(p, grid, stream);
  }
}

}  // namespace

cudaError_t paged_stream4_launch(const StreamParams& p, int head_dim, int row_tile, int grid, cudaStream_t stream) {
  return head_dim == 128 ? launch_d<128>(p, row_tile, grid, stream) : launch_d<64>(p, row_tile, grid, stream);
}

}  // namespace af
