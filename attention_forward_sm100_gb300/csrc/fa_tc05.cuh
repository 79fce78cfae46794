// Persistent, warp-specialised attention forward for sm_103a (tcgen05 + TMA).
//
// Design (prior art: the SM100 flash-attention pages "SM100AttentionSMem",
// "TMAProducerPipeline" and "MHATileScheduler"; rebuilt here for one GB300
// CTA per SM):
//   * a work tile is 256 query rows of one (sequence, head), split into two
//     128-row Q tiles that ping-pong between two softmax warpgroups so the
//     tensor core always has one Q tile's MMAs to run while the other tile's
//     softmax runs (with split-KV, a work tile also names one range of the
//     keys);
//   * warp 14 is the scheduler and the Q/K producer: it takes work indices
//     from an atomic counter (or a static stride, or none: one CTA per work
//     tile), publishes each decoded work tile through a two-slot
//     shared-memory ring (the shared work index of the scheduler page,
//     initial_state / advance) and streams K tiles into a staged ring with
//     TMA and transaction-count mbarriers (acquire / expect-bytes / commit of
//     the producer-pipeline page); warp 15 streams V tiles into their own
//     ring. K is stored k-major and V mn-major (k-major when V is e4m3 and
//     depth-major in memory), all with the 128-byte swizzle, exactly as the
//     MMAs read them;
//   * warps 12 and 13 each issue the tcgen05.mma of one Q tile from one
//     thread: per K/V step one group, O_i += P_i V (P_i read from tensor
//     memory where the softmax left it, over the S_i columns) then
//     S_i = Q_i K^T into tensor memory (fp32); the two issuers' groups
//     strictly alternate through a turn token (the forced-ordering barriers
//     of the layout page);
//   * warpgroups 0 and 1 own Q tiles 0 and 1: thread r owns row r (TMEM lane
//     r), loads S, applies the causal / sequence-end mask, keeps the running
//     max m and sum l in log2 units and writes P = 2^(s*c - m) (bf16, or
//     e4m3 for an e4m3 V) back to tensor memory in two halves. The running
//     max only moves when it grows by more than 2^8, so most tiles need no
//     rescale; when it moves, the softmax warp rescales its own rows of O_i
//     in tensor memory before publishing P. O and l share the max, so O/l is
//     exact;
//   * warpgroup 2 is the epilogue: after the last P V it normalises O by 1/l
//     (handed over through shared memory, the correction region of the
//     layout page), rounds once to bf16 and stores it, or stores the fp32
//     partial row of a split-KV range.
//   * CTA pairs (the pair_cta option of the layout page's barrier set;
//     Tc05Traits<..., PAIR = true>): two CTAs of a cluster on neighbouring
//     SMs share every MMA. A work tile is then 512 rows; each of its two MMA
//     tiles is 256 rows, 128 in each CTA, issued as one M = 256
//     tcgen05.mma.cta_group::2 by the first CTA's issuers. Each CTA loads its
//     own Q rows, half of each K tile (64 keys) and half of each V tile (64
//     depth columns); all copies complete on the first CTA's barriers, the
//     MMA commits arrive in both CTAs (multicast), and the softmax and
//     epilogue warps of the second CTA report to the first CTA's barriers
//     through the cluster window. Work indices are fetched by the first CTA
//     and forwarded to the second through its shared memory.
//   * paged K/V (Tc05Traits<..., PAGED = true>; the newest tokens of each
//     sequence over its paged cache): a K or V tile is gathered page by page
//     (one TMA box per page and 64 depth columns, the page numbers looked up
//     a tile ahead by the producer's lanes), and a 128-row MMA tile packs
//     all (up to 128) query heads that share the KV head times as many tokens
//     as fill it, so each K/V byte that reaches shared memory serves that many
//     heads. The causal mask is aligned to the end of the keys. The slots
//     behind a sequence's last key may hold anything, NaN too: K's are masked
//     as scores, V's are zeroed in shared memory before the tile is handed
//     to the MMAs (a zero weight does not cancel a NaN).
//   * an e4m3 paged cache (Tc05Traits<..., PAGED, C8 = true>): warpgroup 2 also
//     fills the V stages. Its threads copy 16 codes at a time straight from the
//     pages into a two-tile ring (cp.async; every thread reads back only what it
//     copied, so the ring needs no barrier), widen them to bf16 as code * scale,
//     rounded once (exact for powers of two, which is what cache_append
//     writes), and store them where TMA would have put a bf16 tile, zeros
//     behind the sequence's end. With D = 64 K takes the same way. With
//     D = 128 (QSPLIT) K stays e4m3, gathered by TMA, and it is Q that changes:
//     warpgroup 2 writes q = 2^e (q1 + q2) with e4m3 q1 and q2 (a bf16 has
//     eight significant bits, an e4m3 four: q2 takes what q1 leaves, exactly
//     for values above 2^-9 of their row's largest, to 2^-17 of it below: a row's
//     largest is brought to (224, 448], and e4m3's steps end at 2^-9), and
//     S = Q1 K^T + Q2 K^T costs what the bf16 product does. The key scales
//     (copied next to K into a four-tile ring) and 2^e multiply the fp32 scores.
// Every wait is bounded: on timeout the CTA records an error in the
// workspace, raises a shared abort flag that all waits poll (and, in a pair,
// the peer's flag), drains its outstanding copies and MMAs, frees tensor
// memory and exits.
#pragma once
#include <cuda_bf16.h>
#include <math.h>

#include "internal.h"
#include "launch.cuh"
#include "paged.h"
#include "ptx.cuh"
#include "schedule.cuh"

namespace af {

constexpr uint32_t kFull = 0xffffffffu;
constexpr uint64_t kDrainTimeoutNs = 100000000ull;

enum Role : int { kRoleSoftmax0 = 0, kRoleSoftmax1 = 1, kRoleCorrection = 2, kRoleMma = 3, kRoleLoadQK = 4,
                  kRoleLoadV = 5 };

enum BarId : int {
  BAR_Q_FULL = 0,        // +i, TMA transaction barrier of Q tile i
  BAR_Q_EMPTY = 2,       // last S MMA of Q tile 0 done: its Q region is free (tile 1: BAR_Q_EMPTY1)
  BAR_S_FULL = 3,        // +i, S_i = Q_i K^T complete
  BAR_P_LO = 5,          // +i, first half of P_i (keys 0..63) in tensor memory (128 arrivals)
  BAR_STATS = 7,         // +i, final 1/l of Q tile i in shared memory (128 arrivals)
  BAR_P_HI = 9,          // +i, second half of P_i (keys 64..127) in tensor memory (128)
  BAR_O_FINAL = 11,      // +i, last P_i V of a work tile complete
  BAR_O_FREE = 13,       // +i, epilogue finished reading O_i (128)
  BAR_STATS_FREE = 15,   // +i, correction read the 1/l of Q tile i (128)
  BAR_KS = 17,           // +i, fp8 k-scale tile written by the softmax warpgroup (128)
  BAR_SCHED_FULL = 19,   // +slot
  BAR_SCHED_EMPTY = 21,  // +slot
  BAR_DRAIN = 23,        // final commit of the MMA threads
  BAR_ORDER = 24,        // +i, issue turn of MMA issuer i (forced ordering of the two Q tiles)
  BAR_Q_EMPTY1 = 26,     // last S MMA of Q tile 1 done
  BAR_WORK_FULL = 27,    // +slot, CTA pairs: work index written into the second CTA by the first
  BAR_WORK_EMPTY = 29,   // +slot, CTA pairs: the second CTA read that work index
  BAR_SM_TURN = 31,      // +i, softmax turn of warpgroup i (128 arrivals of the other warpgroup)
  BAR_FIXED = 33         // then K_FULL[NK], K_EMPTY[NK], V_FULL[NV], V_EMPTY[NV]
};

constexpr int kScaleSlots = 4;   // tiles of key scales in flight (QSPLIT)
constexpr int kSlotBytes = 48;   // shared-memory bytes of one SchedSlot entry

// Consumers of a scheduler slot: the two MMA lanes, 2 softmax warpgroups, the
// correction warpgroup and the V producer lane.
constexpr uint32_t kSchedConsumers = 2 + 128 + 128 + 128 + 1;

template <int DQK_, int DR_, int DV_, bool FP8_, bool V8_ = false, bool PAIR_ = false, bool PAGED_ = false,
          bool C8_ = false>
struct Tc05Traits {
  static constexpr int DQK = DQK_, DR = DR_, DV = DV_;
  static constexpr bool FP8 = FP8_;
  // e4m3 V, depth-major in global memory: a V stage is Dv rows of 128 keys
  // (K-major B operand of P.V) and P is rounded to e4m3 for kind::f8f6f4.
  static constexpr bool V8 = V8_;
  static_assert(!V8 || (FP8 && DV == 128), "e4m3 V needs e4m3 Q/K and Dv = 128");
  // CTA pair: M = 256 MMAs over two CTAs; this CTA holds 128 of the rows,
  // 64 keys of each K tile and 64 depth columns of each V tile.
  static constexpr bool PAIR = PAIR_;
  static_assert(!PAIR || (!FP8 && DQK == 128 && DV == 128), "CTA pairs: bf16 with Dqk = Dv = 128");
  // K and V gathered from a paged cache, query heads packed into the rows.
  static constexpr bool PAGED = PAGED_;
  static_assert(!PAGED || (!FP8 && !PAIR && DR == 0 && DQK == DV), "paged: bf16 tiles, one CTA, no rope");
  // The paged cache holds e4m3 codes, widened to bf16 on their way to a stage.
  static constexpr bool C8 = C8_;
  static_assert(!C8 || PAGED, "an e4m3 cache is a paged one");
  // K stays e4m3; each Q tile is two e4m3 tiles, q1 and what it leaves, q2.
  static constexpr bool QSPLIT = C8 && DQK == 128;
  static constexpr int BM = kBlockM, BN = kBlockN, NQ = 2;
  static constexpr int MMA_M = PAIR ? 2 * kBlockM : kBlockM;   // rows of one MMA tile (both CTAs)
  static constexpr int ROWS_PER_WORK = NQ * MMA_M;              // rows of one work tile
  static constexpr int QK_CHUNK_ELEMS = FP8 ? 128 : 64;   // elements of one 128-byte swizzle row
  static constexpr int QK_CHUNKS = DQK / QK_CHUNK_ELEMS;
  static constexpr int R_CHUNKS = DR / 64;
  static constexpr int V_CHUNKS = V8 ? 1 : (PAIR ? 1 : DV / 64);   // TMA boxes per V stage (this CTA)
  static constexpr int CHUNK_BYTES = 128 * 128;           // 128 rows x 128 bytes
  static constexpr int K_ROWS = PAIR ? kBlockN / 2 : kBlockN;   // keys of a K stage held by this CTA
  static constexpr int K_CHUNK_BYTES = K_ROWS * 128;
  static constexpr int Q_TILE_BYTES = (QK_CHUNKS + R_CHUNKS) * CHUNK_BYTES;
  static constexpr int K_STAGE_BYTES = QSPLIT ? K_CHUNK_BYTES : (QK_CHUNKS + R_CHUNKS) * K_CHUNK_BYTES;
  static constexpr int V_STAGE_BYTES = V8 ? DV * 128 : V_CHUNKS * CHUNK_BYTES;
  static constexpr int NK = PAIR ? (DR > 0 ? 3 : 5) : (DR > 0 ? 2 : (FP8 ? 4 : (DQK == 64 ? 4 : 3)));
  static constexpr int NV = PAIR ? (DR > 0 ? 3 : 4) : (DR > 0 ? 1 : (V8 ? 4 : (FP8 ? 3 : (DQK == 64 ? 4 : 2))));
  // Bytes one phase of a Q / K / V full barrier waits for (a pair's first CTA
  // counts both CTAs' copies).
  static constexpr uint32_t Q_TX = (PAIR ? 2 : 1) * Q_TILE_BYTES;
  static constexpr uint32_t K_TX = (PAIR ? 2 : 1) * K_STAGE_BYTES;
  static constexpr uint32_t V_TX = (PAIR ? 2 : 1) * V_STAGE_BYTES;

  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = NQ * Q_TILE_BYTES;
  static constexpr int OFF_V = OFF_K + NK * K_STAGE_BYTES;
  static constexpr int OFF_RCPL = OFF_V + NV * V_STAGE_BYTES;       // float [NQ][BM]
  static constexpr int OFF_KS = OFF_RCPL + NQ * BM * 4;             // float [NQ][2][BN] (FP8), [slot][BN] (QSPLIT)
  static constexpr int KS_BYTES = QSPLIT ? kScaleSlots * BN * 4 : (FP8 ? NQ * 2 * BN * 4 : 0);
  static constexpr int OFF_QS = OFF_KS + KS_BYTES;                  // float [NQ][BM] (QSPLIT): 2^e of the rows
  static constexpr int OFF_WIDEN = OFF_QS + (QSPLIT ? NQ * BM * 4 : 0);   // C8: codes and scales of two tiles
  static constexpr int OFF_SCHED = OFF_WIDEN + (C8 ? 2 * (DQK + 4) * BN : 0);               // 2 slots x kSlotBytes
  static constexpr int OFF_WORK = OFF_SCHED + 2 * kSlotBytes;       // CTA pairs: 2 x int64 work index
  static constexpr int OFF_BAR = OFF_WORK + 16;
  static constexpr int NUM_BARS = BAR_FIXED + 2 * NK + 2 * NV + (QSPLIT ? kScaleSlots : (PAGED ? 1 : 0));
  static constexpr int OFF_TMEM_SLOT = OFF_BAR + NUM_BARS * 8;
  static constexpr int OFF_ABORT = OFF_TMEM_SLOT + 4;
  static constexpr int SMEM_BYTES = OFF_ABORT + 12;
  static_assert(SMEM_BYTES <= 232448, "shared memory budget of one CTA exceeded");
  static_assert(OFF_K % 1024 == 0 && OFF_V % 1024 == 0, "swizzled tiles need 1024-byte alignment");

  static constexpr int BAR_K_FULL = BAR_FIXED;
  static constexpr int BAR_K_EMPTY = BAR_FIXED + NK;
  static constexpr int BAR_V_FULL = BAR_FIXED + 2 * NK;
  static constexpr int BAR_V_EMPTY = BAR_FIXED + 2 * NK + NV;
  static constexpr int BAR_V_TAIL = BAR_FIXED + 2 * NK + 2 * NV;   // paged: copies of a V tile that ends inside
  static constexpr int BAR_SCALES = BAR_FIXED + 2 * NK + 2 * NV;   // QSPLIT: +slot, copies of a tile's key scales
  // Arrivals that fill a stage (one per warp of warpgroup 2 where that brings it).
  static constexpr uint32_t Q_FILL = QSPLIT ? 4 : 1, K_FILL = C8 && !QSPLIT ? 4 : 1, V_FILL = C8 ? 4 : 1;

  static constexpr uint32_t TMEM_COLS = 512;
  // Tensor-memory columns: S_0, S_1 (P_i overwrites the first 64 columns of
  // S_i as packed bf16 pairs), O_0, O_1.
  __host__ __device__ static constexpr uint32_t tm_s(int i) { return i ? 128u : 0u; }
  __host__ __device__ static constexpr uint32_t tm_o(int i) { return i ? 384u : 256u; }

  static constexpr uint32_t IDESC_S =
      FP8 || QSPLIT ? ptx::idesc_f32acc(0, 0, false, false, 128, 128) : ptx::idesc_f32acc(1, 1, false, false, MMA_M, 128);
  static constexpr uint32_t IDESC_PV =
      V8 ? ptx::idesc_f32acc(0, 0, false, false, 128, DV) : ptx::idesc_f32acc(1, 1, false, true, MMA_M, DV);
  // P.V instructions per half tile of 64 keys (K = 16 per bf16 instruction, 32 per e4m3).
  static constexpr int PV_INSTR_HALF = V8 ? 2 : 4;
  // TMEM columns of one half of P (64 keys as bf16 pairs or e4m3 quads).
  static constexpr int P_COLS_HALF = V8 ? 16 : 32;
  // MMA instructions of one S = Q K^T (K = 16 per bf16 instruction, 32 per fp8).
  static constexpr int S_INSTR = FP8 ? DQK / 32 : (DQK + DR) / 16;
  // S instructions issued after handing the turn to the other issuer: enough
  // tensor work (~4 x 73 cycles) to cover the other issuer's wake-up.
  static constexpr int S_AFTER_HANDOFF = S_INSTR < 4 ? S_INSTR : 4;

  // Register split (setmaxnreg) of a 512-thread CTA launched with 128 registers per thread.
  // The FP8 softmax (k-scale multiply, e4m3 packing) takes 192 registers; its
  // epilogue warpgroup then fits in 64 (measured: +1-3 % on the FP8
  // workloads, no change for bf16).
    // With an e4m3 cache the epilogue warpgroup also widens K and V (96), and
  // the single-thread roles, which load only Q, get by with 48.
  static constexpr int REG_SOFTMAX = FP8 ? 192 : 184, REG_CORR = FP8 ? 64 : (C8 && !QSPLIT ? 96 : 80),
                       REG_MISC = C8 && !QSPLIT ? 48 : 64;
  // Softmax turn: 0 = the two softmax warpgroups run freely; 1 / 2 = they
  // take turns, handing over after the first half of P / after the tile.
  // With FP8 Q/K a tile's MMAs take less time than a softmax, and two
  // softmaxes that overlap each take twice as long: taking turns keeps them
  // apart.
  static constexpr int SM_TURN = FP8 ? 1 : 0;
  static_assert(2 * 128 * REG_SOFTMAX + 128 * REG_CORR + 128 * REG_MISC <= 512 * 128,
                "register split exceeds the launch allocation");
};

// One decoded work tile as published to every role. With split-KV, k_start
// and lk already describe the tile's own key range. Paged variants: k_start
// and v_start are the first and the end key TILE of the range, lk all keys of
// the sequence, koff the keys in front of its first new token (lk - lq, may be
// negative).
struct SchedSlot {
  int32_t valid, b, h, t, q_start, lq, k_start, lk, split;
  int32_t v_start;   // first key of the tile's range along V's key dimension (packed e4m3 V: own offsets)
  int32_t koff;      // first key of the range within its sequence (0 without split-KV): the causal mask
};

struct Ctx {
  uint8_t* smem;
  uint32_t sbase;
  uint32_t tmem;
  volatile int* abort_flag;
  uint32_t* ws;
  uint64_t timeout_ns;
  int bar_off;
  uint32_t rank;         // CTA pairs: this CTA's rank in the cluster (0 issues the MMAs); else 0
  uint32_t peer_abort;   // CTA pairs: cluster-window address of the peer's abort flag; else 0
  __device__ __forceinline__ uint32_t bar(int i) const { return sbase + bar_off + 8u * (uint32_t)i; }
  // Cluster-window address of barrier i in the pair's first CTA.
  __device__ __forceinline__ uint32_t bar_lead(int i) const { return ptx::mapa(bar(i), 0); }
  __device__ __forceinline__ static int q_empty_id(int i) { return i == 0 ? BAR_Q_EMPTY : BAR_Q_EMPTY1; }
};

__device__ __forceinline__ void raise_error(const Ctx& c, int role, int id) {
  if (atomicCAS(&c.ws[kWsErrorCode], 0u, (uint32_t)kDevErrTimeout) == 0u)
    atomicExch(&c.ws[kWsErrorInfo], ((uint32_t)blockIdx.x << 16) | ((uint32_t)role << 8) | (uint32_t)id);
  *c.abort_flag = 1;
  if (c.peer_abort != 0u) ptx::st_cluster_u32(c.peer_abort, 1u);
}

// Warp-uniform bounded wait: every lane polls, the result is the same in all
// lanes. CLUSTER: the phase completes through arrivals of the peer CTA of a
// pair, whose writes it must see (cluster-scope acquire).
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(const Ctx& c, int id, uint32_t parity, int role) {
  const uint32_t bar = c.bar(id);
  if (__all_sync(kFull, CLUSTER ? ptx::mbar_test_wait_cluster(bar, parity) : ptx::mbar_test_wait(bar, parity)))
    return true;
  const uint64_t t0 = __shfl_sync(kFull, ptx::globaltimer(), 0);
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(kFull, CLUSTER ? ptx::mbar_test_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity)))
      return true;
    if ((it & 63u) == 0u) {
      if (__any_sync(kFull, *c.abort_flag != 0)) return false;
      const uint64_t now = __shfl_sync(kFull, ptx::globaltimer(), 0);
      if (now - t0 > c.timeout_ns) {
        if ((threadIdx.x & 31) == 0) raise_error(c, role, id);
        __syncwarp();
        return false;
      }
    }
  }
}

// Bounded wait of a single thread (the MMA issuers). It polls without ever
// suspending: a thread suspended in mbarrier.try_wait was seen to resume
// hundreds of cycles after the phase completed, and every cycle an issuer
// loses leaves the tensor core idle.
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_one(const Ctx& c, int id, uint32_t parity, int role) {
  const uint32_t bar = c.bar(id);
  auto test = [&]() { return CLUSTER ? ptx::mbar_test_wait_cluster(bar, parity) : ptx::mbar_test_wait(bar, parity); };
  if (test()) return true;
  const uint64_t t0 = ptx::globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (test()) return true;
    if ((it & 255u) == 0u) {
      if (*c.abort_flag != 0) return false;
      if (ptx::globaltimer() - t0 > c.timeout_ns) {
        raise_error(c, role, id);
        return false;
      }
    }
  }
}

// Bounded wait of one thread that ignores the abort flag (drain paths).
__device__ __forceinline__ bool wait_drain(const Ctx& c, int id, uint32_t parity) {
  const uint32_t bar = c.bar(id);
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (ptx::globaltimer() - t0 > kDrainTimeoutNs) return false;
  }
  return true;
}

// CTA pairs: arrival on barrier `id` of the pair's first CTA (a local arrive
// there, a release at cluster scope through the cluster window from the
// second CTA).
__device__ __forceinline__ void arrive_lead(const Ctx& c, int id) {
  if (c.rank == 0) ptx::mbar_arrive(c.bar(id));
  else ptx::mbar_arrive_cluster(c.bar_lead(id));
}

// Ring position: stage index and phase parity.
template <int N>
struct Ring {
  uint32_t idx = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++idx == (uint32_t)N) {
      idx = 0;
      phase ^= 1u;
    }
  }
};

struct Geo {
  int q0;       // first row (within its sequence) of the work tile
  int row[2];   // first row of this CTA's 128 rows of MMA tile i
  int n[2];     // K/V tiles MMA tile i visits
};

template <class T, int CAUSAL>
__device__ __forceinline__ Geo tile_geo(const SchedSlot& s, uint32_t rank, int pack_tokens) {
  Geo g;
  if constexpr (T::PAGED) {
    const int tok = pack_tokens;   // tokens of an MMA tile
    g.q0 = s.t * 2 * tok;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      g.row[i] = g.q0 + tok * i;
      const int kv_end = (CAUSAL & kMaskCausal) ? min(s.lk, s.koff + min(s.lq, g.row[i] + tok)) : s.lk;
      const int end = min(s.v_start, kv_end > 0 ? (kv_end + kBlockN - 1) / kBlockN : 0);
      g.n[i] = max(0, end - s.k_start);
    }
    // Tile 0 visits at least one key tile of a range that tile 1 visits (all
    // of it masked for tile 0): the roles hand over by visited tiles.
    if (g.n[1] > 0 && g.n[0] == 0) g.n[0] = 1;
    return g;
  }
  g.q0 = s.t * T::ROWS_PER_WORK;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    g.row[i] = g.q0 + T::MMA_M * i + kBlockM * (int)rank;
    // causal: keys up to the tile's last row, counted from the range's first key
    const int kv_end = (CAUSAL & kMaskCausal) ? min(s.lk, g.q0 + T::MMA_M * (i + 1) - s.koff) : s.lk;
    g.n[i] = kv_end > 0 ? (kv_end + kBlockN - 1) / kBlockN : 0;
  }
  return g;
}

// Whether this kernel flavour runs split-KV ranges (fixed at compile time;
// the host launches the split flavours exactly when num_splits > 1).
template <int CAUSAL>
__device__ __forceinline__ constexpr bool splits_keys(const Tc05Params&) {
  return (CAUSAL & kMaskNoneSplit) != 0;
}

// Paged variants: the split flavours take their work from a list, in which
// some tiles are cut.
template <int CAUSAL>
__device__ __forceinline__ constexpr bool listed() {
  return (CAUSAL & kMaskNoneSplit) != 0;
}

// The range's key offset travels only in the flavours that use it (causal
// split-KV, paged).
template <int CAUSAL, bool PAGED>
__device__ __forceinline__ SchedSlot read_slot(const Ctx& c, int slot, int off_sched) {
  const volatile int32_t* p = reinterpret_cast<const volatile int32_t*>(c.smem + off_sched + kSlotBytes * slot);
  SchedSlot s;
  s.valid = p[0]; s.b = p[1]; s.h = p[2]; s.t = p[3];
  s.q_start = p[4]; s.lq = p[5]; s.k_start = p[6]; s.lk = p[7]; s.split = p[8]; s.v_start = p[9];
  s.koff = (CAUSAL == kMaskCausalSplit || PAGED) ? p[10] : 0;
  return s;
}

// ---------------------------------------------------------------------------------------------
// Scheduler decode (warp 13, all lanes): work index -> work tile.
struct Cursor {
  int b = 0;
  int64_t base = 0;
};

template <int CAUSAL>
__device__ __forceinline__ SchedSlot decode_work(const Tc05Params& P, int64_t w, Cursor& cur) {
  SchedSlot s;
  s.valid = 0;
  s.b = s.h = s.t = s.q_start = s.k_start = s.split = s.v_start = s.koff = 0;
  s.lq = P.seqlen_q;
  s.lk = P.seqlen_k;
  if (!P.packed) {
    if (w < P.total_work) {
      const WorkTile wt = decode_fixed(w, P.tiles_per_seq, P.num_splits, P.heads_q, P.group, P.kv_chunk);
      s.valid = 1; s.b = wt.b; s.h = wt.h; s.t = wt.t; s.split = wt.split;
      if (splits_keys<CAUSAL>(P)) {
        int32_t j0, j1;
        if (CAUSAL & kMaskCausal)
          causal_split_range(wt.split, P.num_splits, wt.t * P.rows_per_tile, kBlockM, P.rows_per_tile, P.seqlen_k,
                             kBlockN, &j0, &j1);
        else
          split_range(wt.split, P.num_splits, P.kv_tiles, &j0, &j1);
        s.k_start = j0 * kBlockN;
        s.lk = min(P.seqlen_k, j1 * kBlockN) - s.k_start;
        if (CAUSAL == kMaskCausalSplit) s.koff = s.k_start;
      }
      s.v_start = s.k_start;
    }
    return s;
  }
  const int lane = threadIdx.x & 31;
  while (true) {
    const int bb = cur.b + lane;
    int64_t u = 0;
    bool bad = false;
    if (bb < P.batch) {
      // Offsets that would index outside q/k/v/o are refused here, before
      // any use: every sequence passes through this scan in some CTA (the
      // one whose work index runs past the batch scans to its end).
      const int qs = P.cu_q[bb], qe = P.cu_q[bb + 1], ks = P.cu_k[bb], ke = P.cu_k[bb + 1];
      bad = qs < 0 || qe < qs || qe > P.total_q || ks < 0 || ke < ks || ke > P.total_k;
      if (P.cu_v != nullptr) {
        // packed e4m3 V: each sequence's keys start on a 16-key boundary of V
        const int vs = P.cu_v[bb];
        bad = bad || vs < 0 || (vs & 15) != 0 || (int64_t)vs + (ke - ks) > (int64_t)P.total_v;
      }
      if (!bad) u = (int64_t)tiles_for(qe - qs, P.rows_per_tile) * P.heads_q * P.num_splits;
    }
    const unsigned bad_lanes = __ballot_sync(kFull, bad);
    if (bad_lanes) {
      // record it and end this CTA's work (its roles see an invalid slot)
      if (lane == 0 && atomicCAS(&P.ws[kWsErrorCode], 0u, (uint32_t)kDevErrBadSeqlens) == 0u)
        atomicExch(&P.ws[kWsErrorInfo], (uint32_t)(cur.b + __ffs(bad_lanes) - 1));
      return s;
    }
    int64_t incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t n = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += n;
    }
    const unsigned hit = __ballot_sync(kFull, bb < P.batch && w < cur.base + incl);
    if (hit) {
      const int L = __ffs(hit) - 1;
      cur.base += __shfl_sync(kFull, incl - u, L);
      cur.b += L;
      const int b = cur.b;
      const int qs = P.cu_q[b], qe = P.cu_q[b + 1], ks = P.cu_k[b], ke = P.cu_k[b + 1];
      const WorkTile wt = decode_in_sequence(w - cur.base, b, tiles_for(qe - qs, P.rows_per_tile) * P.num_splits,
                                             P.group, P.heads_kv, P.kv_chunk);
      s.valid = 1; s.b = b; s.h = wt.h; s.t = wt.t;
      s.q_start = qs; s.lq = qe - qs; s.k_start = ks; s.lk = ke - ks;
      if (splits_keys<CAUSAL>(P)) {
        // this sequence's own key tiles, cut like the fixed-length case (a
        // range can be empty when the sequence has fewer key tiles than ranges)
        s.split = wt.t % P.num_splits;
        s.t = wt.t / P.num_splits;
        int32_t j0, j1;
        if (CAUSAL & kMaskCausal)
          causal_split_range(s.split, P.num_splits, s.t * P.rows_per_tile, kBlockM, P.rows_per_tile, ke - ks,
                             kBlockN, &j0, &j1);
        else
          split_range(s.split, P.num_splits, tiles_for(ke - ks, kBlockN), &j0, &j1);
        s.k_start = ks + j0 * kBlockN;
        s.lk = min(ke - ks, j1 * kBlockN) - j0 * kBlockN;
        if (CAUSAL == kMaskCausalSplit) s.koff = j0 * kBlockN;
      }
      s.v_start = P.cu_v != nullptr ? P.cu_v[b] + (s.k_start - ks) : s.k_start;
      return s;
    }
    if (cur.b + 32 >= P.batch) return s;
    cur.base += __shfl_sync(kFull, incl, 31);
    cur.b += 32;
  }
}

// The same for a paged problem without a work list: every query tile whole.
// Every sequence has its own number of keys (and of new tokens when packed), so
// the work is found by a scan over the sequences, whose offsets and lengths
// are checked on the way.
template <int CAUSAL>
__device__ __forceinline__ SchedSlot decode_paged(const Tc05Params& P, int64_t w, Cursor& cur) {
  SchedSlot s;
  s.valid = s.b = s.h = s.t = s.q_start = s.lq = s.k_start = s.lk = s.v_start = s.koff = 0;
  s.split = -1;
  const int lane = threadIdx.x & 31;
  const NewRows rows = {P.cu_q, P.seqlens_k, P.batch, P.seqlen_q, P.total_q, P.max_k};
  while (cur.b < P.batch) {
    const int bb = cur.b + lane;
    SeqRows r = {0, 0, 0};
    int64_t u = 0;
    if (bb < P.batch) {
      r = load_seq(rows, bb, P.ws);
      u = (int64_t)tiles_for(r.lq, P.rows_per_tile) * P.heads_q;
    }
    int64_t incl = u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t n = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += n;
    }
    const unsigned hit = __ballot_sync(kFull, bb < P.batch && w < cur.base + incl);
    if (hit) {
      const int L = __ffs(hit) - 1;
      const int64_t first = cur.base + __shfl_sync(kFull, incl - u, L);
      s.b = cur.b + L;
      s.lq = __shfl_sync(kFull, r.lq, L);
      s.lk = __shfl_sync(kFull, r.lk, L);
      s.q_start = __shfl_sync(kFull, r.q0, L);
      const WorkTile wt =
          decode_in_sequence(w - first, s.b, tiles_for(s.lq, P.rows_per_tile), P.group, P.heads_kv, P.kv_chunk);
      s.valid = 1;
      s.h = wt.h;
      s.t = wt.t;
      s.koff = s.lk - s.lq;
      s.v_start = tiles_for(s.lk, kBlockN);
      return s;
    }
    cur.base += __shfl_sync(kFull, incl, 31);
    cur.b += 32;
  }
  return s;
}

// Walk through a work list: items `item` .. `last` belong to the schedule
// entry this CTA has taken.
struct ListCursor {
  int item = 0, last = -1;
  __device__ __forceinline__ bool more() const { return item < last; }
  // The items of schedule entry w (none: item > last).
  __device__ __forceinline__ void take(const Tc05Params& P, int64_t w) {
    const int whole = P.plan->whole;
    item = 0;
    last = -1;
    if (w < whole) {
      item = last = (int)w;
    } else if (w - whole < P.plan->pieces) {
      item = P.pieces[w - whole].first;
      last = P.pieces[w - whole].last;
    }
  }
  __device__ __forceinline__ SchedSlot slot(const Tc05Params& P) const {
    SchedSlot s;
    s.valid = s.b = s.h = s.t = s.q_start = s.lq = s.k_start = s.lk = s.v_start = s.koff = 0;
    s.split = -1;
    if (item <= last) {
      const PlanItem& x = P.items[item];
      s.valid = 1;
      s.b = x.b; s.h = x.h; s.t = x.t;
      s.q_start = x.q_start; s.lq = x.lq; s.lk = x.lk;
      s.k_start = x.j0; s.v_start = x.j1; s.split = x.slot;
      s.koff = x.lk - x.lq;
    }
    return s;
  }
};

// Page of this lane's part of the 128-key tile `tile` of sequence b, -1 if the
// part starts at or past the sequence's end: lane i holds the page of keys
// [i * page_size, (i + 1) * page_size) of the tile (all of it in lane 0's page
// when pages are 128 keys or longer).
__device__ __forceinline__ int tile_page(const Tc05Params& P, const Ctx& c, int b, int lk, int tile) {
  const int lane = threadIdx.x & 31;
  const int key = tile * kBlockN + (lane << P.cache.page_shift);
  if ((lane << P.cache.page_shift) >= kBlockN || key >= lk) return -1;
  return load_page(P.cache, b, key >> P.cache.page_shift, c.ws);
}

// Copies the pages of one K or V tile into a stage (the whole warp; `page` from
// tile_page), completing on `bar`, whose one arrival this is.
template <class T, int CHUNKS>
__device__ __forceinline__ void load_paged_tile(const Tc05Params& P, const CUtensorMap* map, uint32_t dst,
                                                uint32_t bar, int hk, int tile, int page) {
  const int lane = threadIdx.x & 31;
  const int rows = min(kBlockN, 1 << P.cache.page_shift);
  const int parts = __popc(__ballot_sync(kFull, page >= 0));
  if (lane == 0) ptx::mbar_expect_tx(bar, (uint32_t)(parts * rows * 128 * CHUNKS));
  __syncwarp();
  if (page >= 0) {
    const int slot = (tile * kBlockN) & ((1 << P.cache.page_shift) - 1);   // 0 unless pages are longer than a tile
#pragma unroll
    for (int ch = 0; ch < CHUNKS; ++ch)
      ptx::tma_load_4d(dst + ch * T::CHUNK_BYTES + lane * rows * 128, map, bar, ch * 64, hk, slot, page);
  }
  __syncwarp();
}

// Copies the key scales of one tile next to it, into ring slot x (QSPLIT; the
// whole warp, `page` from tile_page). Slot x was last read for tile x - 4: the
// K stage just filled was released by S(x - 3), which followed that softmax.
template <class T>
__device__ __forceinline__ void load_tile_scales(const Tc05Params& P, const Ctx& c, int hk, int tile, int page, uint32_t x) {
  const int lane = threadIdx.x & 31;
  const int rows = min(kBlockN, 1 << P.cache.page_shift);
  const int parts = __popc(__ballot_sync(kFull, page >= 0));
  const uint32_t bar = c.bar(T::BAR_SCALES + (int)(x % kScaleSlots));
  if (lane == 0) ptx::mbar_expect_tx(bar, (uint32_t)(parts * rows * 4));
  __syncwarp();
  if (page >= 0) {
    const int slot = (tile * kBlockN) & ((1 << P.cache.page_shift) - 1);
    const float* src = P.cache.k_scale + ((((int64_t)page * P.cache.heads_kv + hk) << P.cache.page_shift) + slot);
    ptx::bulk_load(c.sbase + T::OFF_KS + (x % kScaleSlots) * (kBlockN * 4) + lane * rows * 4, src, (uint32_t)(rows * 4), bar);
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------------------------
// TMA load of one box into this CTA's shared memory, completing on barrier
// `bar` (in a pair: on that barrier of the pair's first CTA).
template <class T>
__device__ __forceinline__ void load_box(const Ctx& c, uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0,
                                         int c1, int c2, int c3) {
  if constexpr (T::PAIR) ptx::tma_load_4d_pair(dst, map, ptx::mapa(bar, 0), c0, c1, c2, c3);
  else ptx::tma_load_4d(dst, map, bar, c0, c1, c2, c3);
}

// Waits out this CTA's copies in flight after an abort. A pair's second CTA
// cannot watch its copies (they complete on the first CTA's barriers): it
// waits a fixed 200 us, far longer than any copy takes.
__device__ __forceinline__ void pair_copy_grace() {
  const uint64_t t0 = ptx::globaltimer();
  while (ptx::globaltimer() - t0 < 200000ull) {
  }
}

template <class T, int CAUSAL>
__device__ void role_load_qk(const Tc05Params& P, const Ctx& c) {
  const int lane = threadIdx.x & 31;
  const bool lead = c.rank == 0;
  Ring<2> sched;
  Ring<2> fwd;   // CTA pairs: work-index hand-over slots
  Ring<T::NK> kr;
  uint32_t q_empty_phase = 0;
  uint32_t k_fill_parity[T::NK];
  bool k_used[T::NK];
  bool q_loaded[2] = {false, false};
  uint32_t q_fill_parity = 0;
#pragma unroll
  for (int s = 0; s < T::NK; ++s) { k_fill_parity[s] = 0; k_used[s] = false; }
  Cursor cur;
  [[maybe_unused]] ListCursor list;
  [[maybe_unused]] uint32_t sc_tile = 0;   // QSPLIT: key tiles so far
  // The first work index is this CTA's own (a pair's: the cluster's).
  int64_t w = T::PAIR ? (int64_t)ptx::cluster_id_x() : (int64_t)blockIdx.x;
  const int64_t units = T::PAIR ? (int64_t)ptx::nclusters_x() : (int64_t)gridDim.x;
  bool aborted = false;
  while (true) {
    SchedSlot s;
    if constexpr (T::PAGED) {
      if (listed<CAUSAL>()) {
        if (!list.more()) list.take(P, w);
        else ++list.item;
        s = list.slot(P);
      } else {
        s = decode_paged<CAUSAL>(P, w, cur);
      }
    } else {
      s = decode_work<CAUSAL>(P, w, cur);
    }
    if (!wait_warp(c, BAR_SCHED_EMPTY + sched.idx, sched.phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
    if (lane == 0) {
      volatile int32_t* p = reinterpret_cast<volatile int32_t*>(c.smem + T::OFF_SCHED + kSlotBytes * sched.idx);
      p[0] = s.valid; p[1] = s.b; p[2] = s.h; p[3] = s.t;
      p[4] = s.q_start; p[5] = s.lq; p[6] = s.k_start; p[7] = s.lk; p[8] = s.split; p[9] = s.v_start;
      if (CAUSAL == kMaskCausalSplit || T::PAGED) p[10] = s.koff;
      ptx::mbar_arrive(c.bar(BAR_SCHED_FULL + sched.idx));
    }
    __syncwarp();
    sched.next();
    if (!s.valid) break;
    const Geo g = tile_geo<T, CAUSAL>(s, c.rank, P.pack_tokens);
    const int n1 = g.n[1];
    if (n1 > 0) {
      const int hk = s.h / P.group;
      const int qb = P.packed ? 0 : s.b;
      auto load_q = [&](int i) {
        const uint32_t bar = c.bar(BAR_Q_FULL + i);
        const uint32_t dst = c.sbase + T::OFF_Q + i * T::Q_TILE_BYTES;
        const int row = s.q_start + g.row[i];
        // paged: one box is `pack` heads of pack_tokens tokens, 128 rows at most
        if (lead) ptx::mbar_expect_tx(bar, T::PAGED ? (uint32_t)(P.pack * P.pack_tokens * 128 * T::QK_CHUNKS) : T::Q_TX);
        const int head = T::PAGED ? s.h * P.pack : s.h;
#pragma unroll
        for (int ch = 0; ch < T::QK_CHUNKS; ++ch)
          load_box<T>(c, dst + ch * T::CHUNK_BYTES, &P.tm_q, bar, ch * T::QK_CHUNK_ELEMS, head, row, qb);
        if (T::DR > 0) load_box<T>(c, dst + T::QK_CHUNKS * T::CHUNK_BYTES, &P.tm_qr, bar, 0, s.h, row, qb);
      };
      // Q tile 0, K_0, then Q tile 1: each Q region is refilled as soon as
      // its own last S MMA of the previous work tile is done.
      if constexpr (!T::QSPLIT) {   // (else warpgroup 2 brings Q)
        if (!wait_warp(c, BAR_Q_EMPTY, q_empty_phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
        if (lane == 0) load_q(0);
        q_fill_parity = q_empty_phase;   // parity of the Q_FULL phases these loads complete
        q_loaded[0] = true;
        q_loaded[1] = false;
      }
      if constexpr (T::C8 && !T::QSPLIT) {   // warpgroup 2 brings K and V
        if (!wait_warp(c, BAR_Q_EMPTY1, q_empty_phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
        if (lane == 0) load_q(1);
        q_loaded[1] = true;
        q_empty_phase ^= 1u;
      }
      [[maybe_unused]] int page = -1;   // this lane's part of the next K tile
      constexpr bool kLoadsK = !T::C8 || T::QSPLIT;
      if constexpr (T::PAGED && kLoadsK) page = tile_page(P, c, s.b, s.lk, s.k_start);
      for (int j = 0; j < (kLoadsK ? n1 : 0); ++j) {
        if (!wait_warp(c, T::BAR_K_EMPTY + kr.idx, kr.phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
        if constexpr (T::PAGED) {
          load_paged_tile<T, T::K_STAGE_BYTES / T::CHUNK_BYTES>(P, &P.tm_k, c.sbase + T::OFF_K + kr.idx * T::K_STAGE_BYTES,
                             c.bar(T::BAR_K_FULL + kr.idx), hk, s.k_start + j, page);
          if constexpr (T::QSPLIT) {
            load_tile_scales<T>(P, c, hk, s.k_start + j, page, sc_tile);
            ++sc_tile;
          }
          page = tile_page(P, c, s.b, s.lk, s.k_start + j + 1);
        } else if (lane == 0) {
          const uint32_t bar = c.bar(T::BAR_K_FULL + kr.idx);
          const uint32_t dst = c.sbase + T::OFF_K + kr.idx * T::K_STAGE_BYTES;
          // a pair's CTA r holds keys [64 r, 64 r + 64) of the tile
          const int row = s.k_start + kBlockN * j + (T::PAIR ? T::K_ROWS * (int)c.rank : 0);
          if (lead) ptx::mbar_expect_tx(bar, T::K_TX);
#pragma unroll
          for (int ch = 0; ch < T::QK_CHUNKS; ++ch)
            load_box<T>(c, dst + ch * T::K_CHUNK_BYTES, &P.tm_k, bar, ch * T::QK_CHUNK_ELEMS, hk, row, qb);
          if (T::DR > 0) load_box<T>(c, dst + T::QK_CHUNKS * T::K_CHUNK_BYTES, &P.tm_kr, bar, 0, 0, row, qb);
        }
        k_fill_parity[kr.idx] = kr.phase;
        k_used[kr.idx] = true;
        kr.next();
        if (!T::QSPLIT && j == 0) {
          if (!wait_warp(c, BAR_Q_EMPTY1, q_empty_phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
          if (lane == 0) load_q(1);
          q_loaded[1] = true;
          q_empty_phase ^= 1u;
        }
      }
      if (aborted) break;
    }
    // Next work index: from the shared counter (dynamic), one grid stride on
    // (static), or none (one CTA per work tile). A pair's first CTA takes it
    // from the counter and writes it into the second CTA's shared memory.
    if (T::PAGED && listed<CAUSAL>() && list.more()) continue;   // the next segment of this entry
    if (P.schedule == ATTN_SCHEDULE_DYNAMIC) {
      if (!T::PAIR || lead) {
        int64_t nw = 0;
        if (lane == 0) nw = units + (int64_t)atomicAdd(&c.ws[kWsTileCounter], 1u);
        w = __shfl_sync(kFull, nw, 0);
      }
      if constexpr (T::PAIR) {
        const uint32_t slot = c.sbase + T::OFF_WORK + 8u * fwd.idx;
        if (lead) {
          if (!wait_warp<true>(c, BAR_WORK_EMPTY + fwd.idx, fwd.phase ^ 1u, kRoleLoadQK)) { aborted = true; break; }
          if (lane == 0) {
            ptx::st_cluster_u32(ptx::mapa(slot, 1), (uint32_t)(uint64_t)w);
            ptx::st_cluster_u32(ptx::mapa(slot + 4u, 1), (uint32_t)((uint64_t)w >> 32));
            ptx::mbar_arrive_cluster(ptx::mapa(c.bar(BAR_WORK_FULL + fwd.idx), 1));
          }
        } else {
          if (!wait_warp<true>(c, BAR_WORK_FULL + fwd.idx, fwd.phase, kRoleLoadQK)) { aborted = true; break; }
          const volatile uint32_t* ws = reinterpret_cast<const volatile uint32_t*>(c.smem + T::OFF_WORK + 8 * fwd.idx);
          w = (int64_t)(((uint64_t)ws[1] << 32) | (uint64_t)ws[0]);
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive_cluster(c.bar_lead(BAR_WORK_EMPTY + fwd.idx));
        }
        __syncwarp();
        fwd.next();
      }
    } else if (P.schedule == ATTN_SCHEDULE_STATIC) {
      w += units;
    } else {
      w = INT64_MAX;
    }
  }
  if (aborted && lane == 0) {
    if (lead) {
      // Let every copy this warp issued land before the CTA exits.
#pragma unroll
      for (int s = 0; s < T::NK; ++s)
        if (k_used[s]) wait_drain(c, T::BAR_K_FULL + s, k_fill_parity[s]);
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (q_loaded[i]) wait_drain(c, BAR_Q_FULL + i, q_fill_parity);
      if constexpr (T::QSPLIT) {
        for (uint32_t x = sc_tile > kScaleSlots ? sc_tile - kScaleSlots : 0; x < sc_tile; ++x)
          wait_drain(c, T::BAR_SCALES + (int)(x % kScaleSlots), (x / kScaleSlots) & 1u);
      }
    } else {
      pair_copy_grace();
    }
  }
  __syncwarp();
}

template <class T, int CAUSAL>
__device__ void role_load_v(const Tc05Params& P, const Ctx& c) {
  const int lane = threadIdx.x & 31;
  const bool lead = c.rank == 0;
  Ring<2> sched;
  Ring<T::NV> vr;
  uint32_t v_fill_parity[T::NV];
  bool v_used[T::NV];
#pragma unroll
  for (int s = 0; s < T::NV; ++s) { v_fill_parity[s] = 0; v_used[s] = false; }
  bool first_v = true;
  bool aborted = false;
  [[maybe_unused]] uint32_t tail_phase = 0;
  while (true) {
    if (!wait_warp(c, BAR_SCHED_FULL + sched.idx, sched.phase, kRoleLoadV)) { aborted = true; break; }
    const SchedSlot s = read_slot<CAUSAL, T::PAGED>(c, sched.idx, T::OFF_SCHED);
    if (lane == 0) ptx::mbar_arrive(c.bar(BAR_SCHED_EMPTY + sched.idx));
    sched.next();
    if (!s.valid) break;
    const Geo g = tile_geo<T, CAUSAL>(s, c.rank, P.pack_tokens);
    const int hk = s.h / P.group;
    const int vb = P.packed ? 0 : s.b;
    [[maybe_unused]] int page = -1;
    if constexpr (T::PAGED) {
      if (g.n[1] > 0) page = tile_page(P, c, s.b, s.lk, s.k_start);
    }
    for (int j = 0; j < g.n[1]; ++j) {
      if (!wait_warp(c, T::BAR_V_EMPTY + vr.idx, vr.phase ^ 1u, kRoleLoadV)) { aborted = true; break; }
      if constexpr (T::PAGED) {
        const uint32_t dst = c.sbase + T::OFF_V + vr.idx * T::V_STAGE_BYTES;
        const uint32_t full = c.bar(T::BAR_V_FULL + vr.idx);
        const int tile = s.k_start + j, keys = s.lk - tile * kBlockN;
        if (keys >= kBlockN) {
          load_paged_tile<T, T::V_CHUNKS>(P, &P.tm_v, dst, full, hk, tile, page);
          v_used[vr.idx] = true;
        } else {
          // The sequence ends inside this tile: its copies land on a barrier
          // of their own, then the rows behind the end (parts of a page, or
          // whatever the stage held) become zeros.
          load_paged_tile<T, T::V_CHUNKS>(P, &P.tm_v, dst, c.bar(T::BAR_V_TAIL), hk, tile, page);
          if (!wait_warp(c, T::BAR_V_TAIL, tail_phase, kRoleLoadV)) {
            wait_drain(c, T::BAR_V_TAIL, tail_phase);
            aborted = true;
            break;
          }
          tail_phase ^= 1u;
          for (int x = keys * 8 + lane; x < kBlockN * 8; x += 32)
#pragma unroll
            for (int ch = 0; ch < T::V_CHUNKS; ++ch) ptx::st_shared_zero16(dst + ch * T::CHUNK_BYTES + 16 * x);
          ptx::fence_async_shared();   // before the MMAs read what these stores wrote
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(full);
          v_used[vr.idx] = false;      // nothing of this stage is in flight
        }
        v_fill_parity[vr.idx] = vr.phase;
        vr.next();
        page = tile_page(P, c, s.b, s.lk, tile + 1);
        continue;
      }
      // Fault injection (testing only): block 0 never loads its first V tile,
      // so the MMA issuer's bounded wait for it runs out.
      const bool withhold = P.withhold_v && blockIdx.x == 0 && first_v;
      first_v = false;
      if (lane == 0 && !withhold) {
        const uint32_t bar = c.bar(T::BAR_V_FULL + vr.idx);
        const uint32_t dst = c.sbase + T::OFF_V + vr.idx * T::V_STAGE_BYTES;
        const int row = s.k_start + kBlockN * j;
        if (lead) ptx::mbar_expect_tx(bar, T::V_TX);
        if (T::V8) {
          // depth-major e4m3 V: coordinates (key, depth row, head, batch); the
          // key coordinate is a multiple of 16 (a multiple of 128 for fixed
          // length; packed sequences start on 16-key boundaries of V)
          ptx::tma_load_4d(dst, &P.tm_v, bar, s.v_start + kBlockN * j, 0, hk, vb);
        } else if (T::PAIR) {
          // a pair's CTA r holds depth columns [64 r, 64 r + 64) of the tile
          load_box<T>(c, dst, &P.tm_v, bar, 64 * (int)c.rank, hk, row, vb);
        } else {
#pragma unroll
          for (int ch = 0; ch < T::V_CHUNKS; ++ch)
            ptx::tma_load_4d(dst + ch * T::CHUNK_BYTES, &P.tm_v, bar, ch * 64, hk, row, vb);
        }
      }
      v_fill_parity[vr.idx] = vr.phase;
      v_used[vr.idx] = v_used[vr.idx] || !withhold;
      vr.next();
    }
    if (aborted) break;
  }
  if (aborted && lane == 0) {
    if (lead) {
#pragma unroll
      for (int s = 0; s < T::NV; ++s)
        if (v_used[s]) wait_drain(c, T::BAR_V_FULL + s, v_fill_parity[s]);
    } else {
      pair_copy_grace();
    }
  }
  __syncwarp();
}

// ---------------------------------------------------------------------------------------------
// S_i = Q_i K^T, MMA instructions [B, E) of the K loop (nope part first,
// then the shared rope part).
template <class T, int B, int E>
__device__ __forceinline__ void issue_s(const Ctx& c, int i, uint32_t kstage) {
  constexpr uint32_t HI = ptx::sdesc_hi_sw128(1024);
  const uint32_t d = c.tmem + T::tm_s(i);
  const uint32_t qa = ptx::sdesc_lo(ptx::opaque(c.sbase + T::OFF_Q + i * T::Q_TILE_BYTES), 16);
  const uint32_t ka = ptx::sdesc_lo(ptx::opaque(c.sbase + T::OFF_K + kstage * T::K_STAGE_BYTES), 16);
#pragma unroll
  for (int kk = B; kk < E; ++kk) {
    if (T::FP8) {
      ptx::mma_fp8_ss_lo<HI, HI, T::IDESC_S>(d, qa + kk * 2, ka + kk * 2, kk > 0);
    } else if (T::QSPLIT) {   // q1 against the four 32-depth parts of K, then q2
      ptx::mma_fp8_ss_lo<HI, HI, T::IDESC_S>(d, qa + (kk >> 2) * (T::CHUNK_BYTES >> 4) + (kk & 3) * 2, ka + (kk & 3) * 2, kk > 0);
    } else {
      // Q chunks are 128 rows, K chunks K_ROWS rows (64 in a pair)
      const bool rope = kk >= T::DQK / 16;
      const uint32_t qo = (rope ? (T::QK_CHUNKS * T::CHUNK_BYTES + (kk - T::DQK / 16) * 32)
                                : ((kk >> 2) * T::CHUNK_BYTES + (kk & 3) * 32)) >> 4;
      const uint32_t ko = (rope ? (T::QK_CHUNKS * T::K_CHUNK_BYTES + (kk - T::DQK / 16) * 32)
                                : ((kk >> 2) * T::K_CHUNK_BYTES + (kk & 3) * 32)) >> 4;
      if constexpr (T::PAIR) ptx::mma_bf16_ss_lo_pair<HI, HI, T::IDESC_S>(d, qa + qo, ka + ko, kk > 0);
      else ptx::mma_bf16_ss_lo<HI, HI, T::IDESC_S>(d, qa + qo, ka + ko, kk > 0);
    }
  }
}

// O_i += P_i V for keys [64*HALF, 64*HALF + 64) of the tile.
template <class T, int HALF>
__device__ __forceinline__ void issue_pv(const Ctx& c, int i, uint32_t vstage, bool accumulate) {
  constexpr uint32_t HI = ptx::sdesc_hi_sw128(1024);
  const uint32_t d = c.tmem + T::tm_o(i);
  const uint32_t a = c.tmem + T::tm_s(i);   // P: 8 TMEM columns per instruction (16 bf16 / 32 e4m3 keys)
  if (T::V8) {
    // K-major V stage (Dv rows x 128 keys): 32 keys = 32 bytes per instruction
    const uint32_t va = ptx::sdesc_lo(ptx::opaque(c.sbase + T::OFF_V + vstage * T::V_STAGE_BYTES), 16);
#pragma unroll
    for (int kk = 2 * HALF; kk < 2 * HALF + 2; ++kk)
      ptx::mma_fp8_ts_lo<HI, T::IDESC_PV>(d, a + kk * 8, va + kk * 2, (accumulate || kk > 0) ? 1u : 0u);
  } else {
    // MN-major V stage (128 keys x Dv): 16 keys = 2048 bytes per instruction
    const uint32_t va =
        ptx::sdesc_lo(ptx::opaque(c.sbase + T::OFF_V + vstage * T::V_STAGE_BYTES), T::CHUNK_BYTES);
#pragma unroll
    for (int kk = 4 * HALF; kk < 4 * HALF + 4; ++kk) {
      if constexpr (T::PAIR)
        ptx::mma_bf16_ts_lo_pair<HI, T::IDESC_PV>(d, a + kk * 8, va + kk * (2048 >> 4), (accumulate || kk > 0) ? 1u : 0u);
      else
        ptx::mma_bf16_ts_lo<HI, T::IDESC_PV>(d, a + kk * 8, va + kk * (2048 >> 4), (accumulate || kk > 0) ? 1u : 0u);
    }
  }
}

// One MMA-issuing warp per Q tile (warp 12 for tile 0, warp 13 for tile 1).
// Per K/V step g each issues one group, O_i += P_i V_{g-1} then S_i = Q_i K_g^T
// (P_i V first: S_i overwrites the columns holding P_i). The groups of the
// two issuers strictly alternate through a turn token (the forced-ordering
// barriers of the layout page): the tensor core runs tile 0's group while
// tile 1's softmax runs and the other way round. Tile 0, which visits at most
// as many K/V tiles as tile 1, pads with empty groups so that the
// alternation never has to wait for the next work tile. K, V and Q stages are
// released by one commit from each issuer.
// Commit of the issuing thread's MMAs to barrier `id`: in a pair, to that
// barrier in both CTAs (ALL) or in the first CTA only.
template <class T, bool ALL = true>
__device__ __forceinline__ void commit(const Ctx& c, int id) {
  if constexpr (T::PAIR) ptx::mma_commit_pair(c.bar(id), ALL ? (uint16_t)3 : (uint16_t)1);
  else ptx::mma_commit(c.bar(id));
}

template <class T, int CAUSAL>
__device__ void role_mma(const Tc05Params& P, const Ctx& c, const int i) {
  // Runs on lane 0 of warp 12 + i only (in a pair: of the first CTA): one
  // thread issues, waits and commits.
  const int role = kRoleMma;
  Ring<2> sched;
  Ring<T::NK> kr;   // stage of the next K tile
  Ring<T::NV> vr;   // stage of the next V tile
  uint32_t q_full_phase = 0, p_phase = 0, ofree_phase = 0, order_phase = 0;
  // Issuer 0 takes the first turn: its first wait passes on the fresh barrier.
  const uint32_t order_flip = i == 0 ? 1u : 0u;
  bool aborted = false;
#define AF_WAIT(id, par)                   \
  if (!wait_one(c, (id), (par), role)) {   \
    aborted = true;                        \
    break;                                 \
  }
  // barriers that the peer CTA of a pair arrives on
#define AF_WAIT_CL(id, par)                         \
  if (!wait_one<T::PAIR>(c, (id), (par), role)) {   \
    aborted = true;                                 \
    break;                                          \
  }
  while (true) {
    if (!wait_one(c, BAR_SCHED_FULL + sched.idx, sched.phase, role)) { aborted = true; break; }
    const SchedSlot s = read_slot<CAUSAL, T::PAGED>(c, sched.idx, T::OFF_SCHED);
    ptx::mbar_arrive(c.bar(BAR_SCHED_EMPTY + sched.idx));
    sched.next();
    if (!s.valid) break;
    const Geo g = tile_geo<T, CAUSAL>(s, c.rank, P.pack_tokens);
    const int n = g.n[i], n1 = g.n[1];
    if (n1 == 0) {
      // No keys: keep the per-tile O-free handshake in step with the epilogue.
      AF_WAIT_CL(BAR_O_FREE + i, ofree_phase ^ 1u);
      ofree_phase ^= 1u;
      continue;
    }
    AF_WAIT(BAR_Q_FULL + i, q_full_phase);
    q_full_phase ^= 1u;
    for (int grp = 0; grp <= n1; ++grp) {
      const bool has_pv = grp >= 1 && grp <= n;
      const bool has_s = grp < n;
      // Operands that are usually ready first, then the turn, the softmax's
      // first half of P last: once it lands the issuer goes straight to
      // issuing (each barrier check costs this thread ~100-200 cycles while
      // the softmax warps keep tensor and shared memory busy).
      if (has_pv) {
        if (grp == 1) {
          AF_WAIT_CL(BAR_O_FREE + i, ofree_phase ^ 1u);
          ofree_phase ^= 1u;
        }
        AF_WAIT(T::BAR_V_FULL + vr.idx, vr.phase);
      }
      if (has_s) AF_WAIT(T::BAR_K_FULL + kr.idx, kr.phase);
      if (!wait_one(c, BAR_ORDER + i, order_phase ^ order_flip, role)) { aborted = true; break; }
      order_phase ^= 1u;
      if (has_pv) AF_WAIT_CL(BAR_P_LO + i, p_phase);
      ptx::tc_fence_after();
      if (has_pv) {
        issue_pv<T, 0>(c, i, vr.idx, grp > 1);
        AF_WAIT_CL(BAR_P_HI + i, p_phase);
        p_phase ^= 1u;
        ptx::tc_fence_after();
        issue_pv<T, 1>(c, i, vr.idx, true);
        commit<T>(c, T::BAR_V_EMPTY + vr.idx);
        if (grp == n) commit<T>(c, BAR_O_FINAL + i);
        vr.next();
      }
      if (has_s) {
        // Hand the turn over before the last S_AFTER_HANDOFF instructions, so
        // the other issuer's wake-up overlaps their execution.
        issue_s<T, 0, T::S_INSTR - T::S_AFTER_HANDOFF>(c, i, kr.idx);
        ptx::mbar_arrive(c.bar(BAR_ORDER + (i ^ 1)));
        issue_s<T, T::S_INSTR - T::S_AFTER_HANDOFF, T::S_INSTR>(c, i, kr.idx);
        commit<T>(c, BAR_S_FULL + i);
        commit<T>(c, T::BAR_K_EMPTY + kr.idx);
        if (grp == n - 1) commit<T>(c, Ctx::q_empty_id(i));
        kr.next();
      } else {
        ptx::mbar_arrive(c.bar(BAR_ORDER + (i ^ 1)));   // the other issuer's turn
      }
      if (!has_pv && !has_s) {
        // A K/V tile only the other Q tile visits: release this issuer's share.
        AF_WAIT(T::BAR_K_FULL + kr.idx, kr.phase);
        commit<T>(c, T::BAR_K_EMPTY + kr.idx);
        kr.next();
        AF_WAIT(T::BAR_V_FULL + vr.idx, vr.phase);
        commit<T>(c, T::BAR_V_EMPTY + vr.idx);
        vr.next();
      }
    }
    if (aborted) break;
  }
#undef AF_WAIT
#undef AF_WAIT_CL
  // Drain: the arrive of this commit follows every MMA and commit this thread
  // issued (both issuers commit; the phase completes after both).
  commit<T, false>(c, BAR_DRAIN);
  wait_drain(c, BAR_DRAIN, 0);
  (void)aborted;
}

// ---------------------------------------------------------------------------------------------
// Paged variants: row r of an MMA tile as token and head of the tile; the rows
// behind pack_tokens * pack belong to nobody.
struct PackedRow {
  int tok, h;
  bool ok;
  __device__ __forceinline__ PackedRow(const Tc05Params& P, int r) {
    tok = P.pack > 0 ? r / P.pack : r;
    h = r - tok * P.pack;
    ok = tok < P.pack_tokens;
  }
};

// Paged variants: LSE element of token qi and query head h.
__device__ __forceinline__ int64_t paged_lse_index(const Tc05Params& P, const SchedSlot& s, int qi, int h) {
  return P.packed ? (int64_t)h * P.total_q + s.q_start + qi : ((int64_t)s.b * P.heads_total + h) * P.seqlen_q + qi;
}

template <class T, int CAUSAL>
__device__ void role_softmax(const Tc05Params& P, const Ctx& c, const int i) {
  const int tid = threadIdx.x - 128 * i;          // row of the Q tile == TMEM lane
  const uint32_t lane_base = (uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16;
  const uint32_t tS = c.tmem + lane_base + T::tm_s(i);
  const uint32_t tO = c.tmem + lane_base + T::tm_o(i);
  float* rcpl_sm = reinterpret_cast<float*>(c.smem + T::OFF_RCPL) + i * kBlockM;
  float* ks_sm = reinterpret_cast<float*>(c.smem + T::OFF_KS) + i * 2 * kBlockN;
  const int role = i == 0 ? kRoleSoftmax0 : kRoleSoftmax1;
  [[maybe_unused]] const PackedRow pk(P, tid);
  Ring<2> sched;
  uint32_t s_phase = 0, ks_phase = 0, stats_phase = 0, turn_phase = 0;
  [[maybe_unused]] uint32_t q_phase = 0, sc_tile = 0;   // QSPLIT (sc_tile: key tiles before this work tile's)
  const uint32_t turn_flip = i == 0 ? 1u : 0u;   // warpgroup 0 takes the first turn
  while (true) {
    if (!wait_warp(c, BAR_SCHED_FULL + sched.idx, sched.phase, role)) return;
    const SchedSlot s = read_slot<CAUSAL, T::PAGED>(c, sched.idx, T::OFF_SCHED);
    ptx::mbar_arrive(c.bar(BAR_SCHED_EMPTY + sched.idx));
    sched.next();
    if (!s.valid) return;
    const Geo g = tile_geo<T, CAUSAL>(s, c.rank, P.pack_tokens);
    const int n = g.n[i];
    const int qi = T::PAGED ? g.row[i] + pk.tok : g.row[i] + tid;   // row within the sequence
    const bool row_valid = qi < s.lq && (!T::PAGED || pk.ok);
    // keys of the range visible to this row (causal: keys 0..qi of the
    // sequence, the range starting at key koff of it)
    // (paged: keys 0 .. koff + qi, the range starting at key tile k_start)
    int lim, klen, first_row;   // visible keys, keys of the range, first row's last key in the range
    if constexpr (T::PAGED) {
      klen = s.lk - s.k_start * kBlockN;
      lim = (CAUSAL & kMaskCausal) ? min(klen, s.koff + qi + 1 - s.k_start * kBlockN) : klen;
      first_row = s.koff + g.row[i] - s.k_start * kBlockN;
    } else {
      klen = s.lk;
      lim = (CAUSAL & kMaskCausal) ? min(s.lk, qi + 1 - s.koff) : s.lk;
      first_row = g.row[i] - s.koff;
    }
    // LSE element: [B][Hq][Sq] (or [Hq][Tq] packed); a split-KV range writes
    // its partial LSE to copy `split` of that layout, [split][B][Hq][Sq] (or
    // [split][Hq][Tq]).
    const bool split_kv = splits_keys<CAUSAL>(P);
    const int sp = split_kv ? s.split : 0;
    const bool partial = T::PAGED ? listed<CAUSAL>() && s.split >= 0 : splits_keys<CAUSAL>(P);
    const int64_t lse_idx = T::PAGED ? (partial ? (int64_t)s.split * kRowsPerTile + kBlockM * i + tid
                                                : paged_lse_index(P, s, qi, s.h * P.pack + pk.h))
                          : P.packed ? ((int64_t)sp * P.heads_q + s.h) * P.total_q + s.q_start + qi
                                     : (((int64_t)sp * P.batch + s.b) * P.heads_q + s.h) * P.seqlen_q + qi;
    float c_row = P.scale_log2;
    int64_t ks_base = 0;
    if (T::FP8) {
      const int hk = s.h / P.group;
      float qs = 1.f;
      if (row_valid)
        qs = P.packed ? P.q_scale[(int64_t)s.h * P.total_q + s.q_start + qi]
                      : P.q_scale[((int64_t)s.b * P.heads_q + s.h) * P.seqlen_q + qi];
      c_row *= qs;
      ks_base = P.packed ? (int64_t)hk * P.total_k + s.k_start
                         : ((int64_t)s.b * P.heads_kv + hk) * P.seqlen_k + s.k_start;
    }
    float ks_next = 0.f;
    if constexpr (T::QSPLIT) {
      if (n > 0) {
        // Warpgroup 2 wrote this work tile's row factors before it filled Q; it
        // writes the next ones after this warpgroup's statistics.
        if (!wait_warp(c, BAR_Q_FULL + i, q_phase, role)) return;
        c_row *= reinterpret_cast<const float*>(c.smem + T::OFF_QS)[kBlockM * i + tid];
      }
      if (g.n[1] > 0) q_phase ^= 1u;
    }
    if (T::FP8 && n > 0) ks_next = tid < s.lk ? __ldg(P.k_scale + ks_base + tid) : 0.f;
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < n; ++j) {
      const int kb = kBlockN * j;
      if (T::FP8) {
        ks_sm[(j & 1) * kBlockN + tid] = ks_next;
        ptx::mbar_arrive(c.bar(BAR_KS + i));
        if (!wait_warp(c, BAR_KS + i, ks_phase, role)) return;
        ks_phase ^= 1u;
        if (j + 1 < n) ks_next = (kb + kBlockN + tid < s.lk) ? __ldg(P.k_scale + ks_base + kb + kBlockN + tid) : 0.f;
      }
      if (!wait_warp(c, BAR_S_FULL + i, s_phase, role)) return;
      s_phase ^= 1u;
      if (T::SM_TURN) {
        if (!wait_warp(c, BAR_SM_TURN + i, turn_phase ^ turn_flip, role)) return;
        turn_phase ^= 1u;
      }
      ptx::tc_fence_after();
      float sv[128];
      {
        uint32_t r[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) ptx::tmem_ld32(tS + 32 * q, r[q]);
        ptx::tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[32 * q + e] = __uint_as_float(r[q][e]);
      }
      if constexpr (T::QSPLIT) {
        // The slot's copies are complete (S needed K, and a slot is refilled only
        // once the S after next is done): the wait makes them visible here.
        const uint32_t x = sc_tile + (uint32_t)j;
        if (!wait_warp(c, T::BAR_SCALES + (int)(x % kScaleSlots), (x / kScaleSlots) & 1u, role)) return;
        const float4* k4 = reinterpret_cast<const float4*>(c.smem + T::OFF_KS) + (x % kScaleSlots) * (kBlockN / 4);
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float4 kv = k4[e];
          ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(sv[4 * e], sv[4 * e + 1]), ptx::f2_pack(kv.x, kv.y)), sv[4 * e],
                         sv[4 * e + 1]);
          ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(sv[4 * e + 2], sv[4 * e + 3]), ptx::f2_pack(kv.z, kv.w)),
                         sv[4 * e + 2], sv[4 * e + 3]);
        }
      }
      if (T::FP8) {
        const float2* k2 = reinterpret_cast<const float2*>(ks_sm + (j & 1) * kBlockN);
#pragma unroll
        for (int e = 0; e < 64; ++e) {
          const float2 kv = k2[e];
          float a0, a1;
          ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(sv[2 * e], sv[2 * e + 1]), ptx::f2_pack(kv.x, kv.y)), a0, a1);
          sv[2 * e] = a0;
          sv[2 * e + 1] = a1;
        }
      }
      const bool need_mask = (kb + kBlockN > klen) || ((CAUSAL & kMaskCausal) && kb + kBlockN - 1 > first_row);
      if (need_mask) {
        const int vis = lim - kb;
        if constexpr (T::V8) {
          // one compare per key (measured 5 % faster here than the per-chunk
          // bit pattern below, which is ~1 % faster in the other variants)
#pragma unroll
          for (int e = 0; e < 128; ++e)
            if (e >= vis) sv[e] = -INFINITY;
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int vq = min(max(vis - 32 * q, 0), 32);
            const uint32_t bits = vq >= 32 ? 0xffffffffu : ((1u << vq) - 1u);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!((bits >> e) & 1u)) sv[32 * q + e] = -INFINITY;
          }
        }
      }
      float mx0 = ptx::max3(sv[0], sv[1], sv[2]), mx1 = ptx::max3(sv[3], sv[4], sv[5]);
      float mx2 = ptx::max3(sv[6], sv[7], sv[8]), mx3 = ptx::max3(sv[9], sv[10], sv[11]);
#pragma unroll
      for (int e = 12; e < 124; e += 8) {
        mx0 = ptx::max3(mx0, sv[e], sv[e + 1]);
        mx1 = ptx::max3(mx1, sv[e + 2], sv[e + 3]);
        mx2 = ptx::max3(mx2, sv[e + 4], sv[e + 5]);
        mx3 = ptx::max3(mx3, sv[e + 6], sv[e + 7]);
      }
      mx0 = ptx::max3(mx0, sv[124], sv[125]);
      mx1 = ptx::max3(mx1, sv[126], sv[127]);
      const float mx = ptx::max3(mx0, mx1, fmaxf(mx2, mx3)) * c_row;
      const float m_new = fmaxf(m, mx);
      float m_use = m, alpha = 1.f;
      if (j == 0) {
        m_use = m_new;
      } else if (m_new > m + 8.f) {
        m_use = m_new;
        alpha = ptx::ex2(m - m_new);
      }
      const uint64_t c2 = ptx::f2_pack(c_row, c_row);
      // paged: a row may see no key of a tile it visits; its maximum stays -inf
      // and its weights are 0, not exp(-inf + inf)
      const float neg = T::PAGED && m_use == -INFINITY ? 0.f : -m_use;
      const uint64_t n2 = ptx::f2_pack(neg, neg);
      uint64_t acc0 = 0, acc1 = 0;   // (+0.0f, +0.0f) pairs
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        // P for keys [64*half, 64*half + 64) -> 32 packed bf16 pairs (or 16
        // e4m3 quads).
        uint32_t pk[T::P_COLS_HALF];
        [[maybe_unused]] float q0 = 0.f, q1 = 0.f;   // e4m3: the previous pair of the quad
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int el = 64 * half + 2 * e;
          float x0, x1;
          ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(sv[el], sv[el + 1]), c2, n2), x0, x1);
          const float p0 = ptx::ex2(x0), p1 = ptx::ex2(x1);
          if (e & 1) acc1 = ptx::f2_add(acc1, ptx::f2_pack(p0, p1));
          else acc0 = ptx::f2_add(acc0, ptx::f2_pack(p0, p1));
          if constexpr (T::V8) {
            if (e & 1) pk[e >> 1] = ptx::pack_e4m3x4(q0, q1, p0, p1);
            q0 = p0;
            q1 = p1;
          } else {
            pk[e] = ptx::pack_bf16(p0, p1);
          }
        }
        if constexpr (T::V8) ptx::tmem_st16(tS + T::P_COLS_HALF * half, pk);
        else ptx::tmem_st32(tS + T::P_COLS_HALF * half, pk);
        if (half == 0 && __any_sync(kFull, alpha != 1.f)) {
          // Correction: the running max moved (rare with the 2^8 headroom), so
          // rescale this warp's rows of O_i before the next P V accumulates
          // into it. P_i(j-1) V was complete when S_i(j) arrived (same issuer,
          // in order).
#pragma unroll 1
          for (int q = 0; q < T::DV / 32; ++q) {
            uint32_t r[32];
            ptx::tmem_ld32(tO + 32 * q, r);
            ptx::tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            ptx::tmem_st32(tO + 32 * q, r);
          }
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before();
        if constexpr (T::PAIR) {
          // one arrival per warp on the first CTA's barrier
          __syncwarp();
          if ((threadIdx.x & 31) == 0) arrive_lead(c, (half == 0 ? BAR_P_LO : BAR_P_HI) + i);
        } else {
          ptx::mbar_arrive(c.bar((half == 0 ? BAR_P_LO : BAR_P_HI) + i));
        }
        if (T::SM_TURN == half + 1) ptx::mbar_arrive(c.bar(BAR_SM_TURN + (i ^ 1)));   // the other warpgroup's turn
      }
      float s0, s1, s2, s3;
      ptx::f2_unpack(acc0, s0, s1);
      ptx::f2_unpack(acc1, s2, s3);
      l = l * alpha + ((s0 + s1) + (s2 + s3));
      m = m_use;
    }
    if constexpr (T::QSPLIT) sc_tile += (uint32_t)g.n[1];
    if (T::SM_TURN) {
      // K/V tiles only the other Q tile visits: pass the turn on.
      for (int j = n; j < g.n[1]; ++j) {
        if (!wait_warp(c, BAR_SM_TURN + i, turn_phase ^ turn_flip, role)) return;
        turn_phase ^= 1u;
        ptx::mbar_arrive(c.bar(BAR_SM_TURN + (i ^ 1)));
      }
    }
    // Row statistics: LSE (natural log) here, 1/l to the epilogue. A split-KV
    // range writes the LSE of its own keys for the merge.
    float* const lse_dst = partial ? P.lse_part : P.lse;
    // (paged: a row with a NaN score is NaN, not one that sees nothing)
    const bool some = T::PAGED ? l != 0.f : l > 0.f;
    if (row_valid && lse_dst != nullptr) {
      const float lse = some ? (m + ptx::lg2(l)) * 0.69314718055994531f : -INFINITY;
      lse_dst[lse_idx] = lse;
    }
    if (!wait_warp(c, BAR_STATS_FREE + i, stats_phase ^ 1u, role)) return;
    stats_phase ^= 1u;
    rcpl_sm[tid] = some ? 1.f / l : 0.f;
    ptx::mbar_arrive(c.bar(BAR_STATS + i));
  }
}

// ---------------------------------------------------------------------------------------------
// 32 columns of one O row (64 bytes) as bf16: two 32-byte stores when O is
// 32-byte aligned (whole sectors per instruction), else four 16-byte ones.
template <class T>
__device__ __forceinline__ void store_row_chunk(uint16_t* dst, const uint32_t (&r)[32], float scale, bool wide) {
  uint32_t pk[16];
#pragma unroll
  for (int e = 0; e < 16; ++e)
    pk[e] = ptx::pack_bf16(__uint_as_float(r[2 * e]) * scale, __uint_as_float(r[2 * e + 1]) * scale);
  if (wide) {
    ptx::st_global_v8(dst, pk);
    ptx::st_global_v8(dst + 16, pk + 8);
  } else {
    uint4* d = reinterpret_cast<uint4*>(dst);
#pragma unroll
    for (int e = 0; e < 4; ++e) d[e] = make_uint4(pk[4 * e], pk[4 * e + 1], pk[4 * e + 2], pk[4 * e + 3]);
  }
}

// Split-KV: row of the partial O array [split][rows][Hq] (rows = B*Sq, or Tq
// when packed) of query row qi of work tile s.
__device__ __forceinline__ int64_t partial_row(const Tc05Params& P, const SchedSlot& s, int qi) {
  const int64_t rows = P.packed ? (int64_t)P.total_q : (int64_t)P.batch * P.seqlen_q;
  const int64_t row = P.packed ? (int64_t)s.q_start + qi : (int64_t)s.b * P.seqlen_q + qi;
  return ((int64_t)s.split * rows + row) * P.heads_q + s.h;
}

// Split-KV: one 32-column chunk of a row of normalised partial O, in fp32,
// as four 32-byte stores (partial rows are 32-byte aligned in the workspace).
__device__ __forceinline__ void store_row_chunk_f32(float* dst, const uint32_t (&r)[32], float scale) {
  uint32_t v[32];
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(r[e]) * scale);
#pragma unroll
  for (int e = 0; e < 4; ++e) ptx::st_global_v8(dst + 8 * e, v + 8 * e);
}

// ---------------------------------------------------------------------------------------------
// C8: warpgroup 2 as the V producer (QSPLIT; else of K and V). A unit is one K or
// V tile, 128 rows of D codes; warp w brings rows 32 w .. 32 w + 31, D / 16 lanes to a row (16 codes
// each), in D / 16 pieces per thread. The pieces of unit u go through half
// u & 1 of a ring, each refilled with unit u + 2's as soon as it is read: two
// units (32 KB at D = 128) are in flight, a whole step's bytes. (Registers in
// place of the ring hold one unit: 2048 new tokens behind 30720, GQA 32/8, took
// 1394 us with them and 1305 with the ring, the rest being the same.) In every
// pair of rows the lanes of the upper 64 depths take the other row: the two
// 16-byte halves that a lane stores then fall on different banks across its
// eight neighbours.
template <class T>
struct Widen {
  static constexpr int LPR = T::DQK / 16;        // lanes per row
  static constexpr int RPL = 32 / LPR;           // rows a warp moves at a time
  static constexpr int NP = 32 / RPL;            // pieces per thread
  static constexpr int PB = 16 / RPL;            // of them in a 16-key block
  static constexpr int RING = T::OFF_WIDEN;      // [2][NP][128 threads][16 bytes]
  static constexpr int SCALES = T::OFF_WIDEN + 2 * NP * 2048;   // [2][128 rows] fp32

  Ring<T::NK> kr;
  Ring<T::NV> vr;

  __device__ static int row0() {   // this lane's first row of a unit
    const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31, col = lane % LPR;
    return 32 * w + ((lane / LPR) ^ (T::DQK == 128 && col >= 4 ? 1 : 0));
  }
  // Byte offset in a stage of this lane's first 8 values of piece 0; the other
  // 8 follow at ^ 16, piece i RPL rows on (the swizzle is the row modulo 8).
  __device__ static uint32_t lane_offset() {
    const int col = (threadIdx.x & 31) % LPR, r = row0();
    return ((2 * col) >> 3) * T::CHUNK_BYTES + r * 128 + ((((2 * col) & 7) ^ (r & 7)) << 4);
  }
  // 16 codes of piece i times their scale as bf16 at `at` (stage + lane_offset).
  __device__ static __forceinline__ void store(uint32_t at, int i, const uint4& v, float scale) {
    const uint32_t a = (RPL == 4 && (i & 1) ? at ^ 64u : at) + i * RPL * 128;
    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
    uint32_t y[8];
    const uint64_t s2 = ptx::f2_pack(scale, scale);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      uint32_t h[2];
      ptx::e4m3x4_to_f16x2(x[e >> 1], h[0], h[1]);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float lo, hi;
        ptx::f16x2_to_float2(h[k], lo, hi);
        ptx::f2_unpack(ptx::f2_mul(ptx::f2_pack(lo, hi), s2), lo, hi);
        y[e + k] = ptx::pack_bf16(lo, hi);
      }
    }
    ptx::st_shared_v4(a, y[0], y[1], y[2], y[3]);
    ptx::st_shared_v4(a ^ 16u, y[4], y[5], y[6], y[7]);
  }

  // Where this thread's pieces of a unit come from.
  struct Source {
    const uint8_t *lo, *hi;  // this lane's first row in the two 16-key blocks of its warp's rows
    int64_t step;            // bytes between its rows of a block
    int keys;                // rows from its first one to the sequence's end
  };
  __device__ static __forceinline__ Source aim(const CacheView& cv, const uint8_t* base, int64_t page_stride,
                                               int64_t tok, const int (&page)[2], int tile, int lk) {
    const int r0 = row0(), at = tile * kBlockN + r0, mask = (1 << cv.page_shift) - 1;
    base += ((threadIdx.x & 31) % LPR) * 16;
    Source s;
    s.keys = lk - at;
    s.step = tok * RPL;
    s.lo = base + page[0] * page_stride + (int64_t)(at & mask) * tok;
    s.hi = base + page[1] * page_stride + (int64_t)((at + 16) & mask) * tok;
    return s;
  }
  // Copy of piece i to `dst`; zeros behind the end.
  __device__ static __forceinline__ void copy(const CacheView& cv, const Source& s, uint32_t dst, int i) {
    const bool ok = RPL * i < s.keys;
    const uint8_t* row = i < PB ? s.lo + i * s.step : s.hi + (i - PB) * s.step;
    ptx::cp_async16(dst, ok ? row : cv.k, ok);
  }
  // Copy of the scale of row (thread) of a unit.
  __device__ static __forceinline__ void copy_scale(const Ctx& c, const CacheView& cv, const float* scales, int hk,
                                                    const int (&page)[2], int tile, int lk, uint32_t half) {
    const int tid = threadIdx.x & 127, key = tile * kBlockN + tid;
    const bool ok = key < lk;
    const int64_t at = (((int64_t)page[(tid >> 4) & 1] * cv.heads_kv + hk) << cv.page_shift) +
                       (key & ((1 << cv.page_shift) - 1));
    ptx::cp_async4(c.sbase + SCALES + half * 512 + tid * 4, ok ? scales + at : scales, ok);
  }
  // All units of one work tile, the first two on their way since begin():
  // K_0, V_0, K_1, V_1, ... or, with QSPLIT, V_0, V_1, ... False: a wait ran out.
  // One small loop, unrolled twice only: with the code of every piece laid out,
  // this warpgroup and the softmax ones evicted each other's instructions.
  static constexpr bool BOTH = !T::QSPLIT;
  __device__ static __forceinline__ bool is_v(int u) { return BOTH ? (u & 1) != 0 : true; }
  __device__ static __forceinline__ int tile_of(int u) { return BOTH ? u >> 1 : u; }
  __device__ static __forceinline__ void pages_of(const Tc05Params& P, const Ctx& c, const SchedSlot& s, int tile,
                                                  int (&page)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = (s.k_start + tile) * kBlockN + 32 * ((threadIdx.x >> 5) & 3) + 16 * h;
      page[h] = key < s.lk ? load_page(P.cache, s.b, key >> P.cache.page_shift, c.ws) : 0;
    }
  }
  __device__ static __forceinline__ Source source(const Tc05Params& P, const SchedSlot& s, int u, int hk,
                                                  const int (&page)[2]) {
    const CacheView& cv = P.cache;
    return is_v(u) ? aim(cv, cv.v + hk * cv.v_head, cv.v_page, cv.v_tok, page, s.k_start + tile_of(u), s.lk)
                   : aim(cv, cv.k + hk * cv.k_head, cv.k_page, cv.k_tok, page, s.k_start + tile_of(u), s.lk);
  }
  __device__ __forceinline__ void begin(const Tc05Params& P, const Ctx& c, const SchedSlot& s, int n) {
    const int hk = s.h / P.group;
    const uint32_t ring0 = c.sbase + RING + (threadIdx.x & 127) * 16;
    int page[2];
#pragma unroll 1
    for (int u = 0; u < 2; ++u) {
      if (u == 0 || !BOTH) pages_of(P, c, s, tile_of(u), page);   // (past the end: pages 0, nothing is read)
      const Source src = source(P, s, u, hk, page);
#pragma unroll
      for (int i = 0; i < NP; ++i) copy(P.cache, src, ring0 + (u * NP + i) * 2048, i);
      copy_scale(c, P.cache, is_v(u) ? P.cache.v_scale : P.cache.k_scale, hk, page, s.k_start + tile_of(u), s.lk, u);
      ptx::cp_async_commit();
    }
  }
  __device__ __forceinline__ bool run(const Tc05Params& P, const Ctx& c, const SchedSlot& s, int n) {
    const int lane = threadIdx.x & 31;
    const int hk = s.h / P.group;
    const CacheView& cv = P.cache;
    const int units = BOTH ? 2 * n : n;
    const uint32_t at0 = c.sbase + lane_offset();
    const uint32_t ring0 = c.sbase + RING + (threadIdx.x & 127) * 16;
    int page[2];   // of unit u + 2's tile
    pages_of(P, c, s, tile_of(2), page);
#pragma unroll 1
    for (int u = 0; u < units; ++u) {
      const uint32_t half = u & 1;
      const bool v = is_v(u);
      Source next = source(P, s, u + 2, hk, page);
      if (u + 2 >= units) next.keys = 0;            // (zeros, read by nobody)
      const int empty = v ? T::BAR_V_EMPTY + (int)vr.idx : T::BAR_K_EMPTY + (int)kr.idx;
      if (!wait_warp(c, empty, (v ? vr.phase : kr.phase) ^ 1u, v ? kRoleLoadV : kRoleLoadQK)) {
        ptx::cp_async_wait<0>();
        return false;
      }
      ptx::cp_async_wait<1>();
      __syncwarp();   // the scales were copied by other lanes
      const uint32_t at = at0 + (v ? T::OFF_V + vr.idx * T::V_STAGE_BYTES : T::OFF_K + kr.idx * T::K_STAGE_BYTES);
      const uint32_t ring = ring0 + half * NP * 2048;
      const float* sc = reinterpret_cast<const float*>(c.smem + SCALES + half * 512) + row0();
#pragma unroll 1
      for (int i = 0; i < NP; i += 2) {
        const uint4 v0 = ptx::ld_shared_v4(ring + i * 2048), v1 = ptx::ld_shared_v4(ring + i * 2048 + 2048);
        const float s0 = sc[RPL * i], s1 = sc[RPL * i + RPL];
        store(at + i * RPL * 128, 0, v0, s0);
        store(at + i * RPL * 128, 1, v1, s1);
        copy(cv, next, ring + i * 2048, i);
        copy(cv, next, ring + i * 2048 + 2048, i + 1);
      }
      ptx::fence_async_shared();   // before the MMAs read the stage
      __syncwarp();
      if (v) {
        if (lane == 0) ptx::mbar_arrive(c.bar(T::BAR_V_FULL + vr.idx));
        vr.next();
      } else {
        if (lane == 0) ptx::mbar_arrive(c.bar(T::BAR_K_FULL + kr.idx));
        kr.next();
      }
      copy_scale(c, cv, v ? cv.v_scale : cv.k_scale, hk, page, s.k_start + tile_of(u + 2), u + 2 < units ? s.lk : 0, half);
      ptx::cp_async_commit();
      if (v) pages_of(P, c, s, tile_of(u + 3), page);   // (the same tile's V follows its K)
    }
    ptx::cp_async_wait<0>();
    return true;
  }
};

// QSPLIT: Q tile i of a work tile from global memory into its two e4m3 tiles, one
// row per thread (warpgroup 2): with s the smallest power of two that brings the
// row to 448 or below, q1 = e4m3(q / s), q2 = e4m3(q / s - q1), and s for the
// softmax. Rows behind the sequence are zeros.
template <class T>
__device__ __forceinline__ void split_q(const Tc05Params& P, const Ctx& c, const SchedSlot& s, int first, int i) {
  const int r = threadIdx.x & 127;
  const PackedRow pk(P, r);
  const int tok = first + pk.tok, h = s.h * P.pack + pk.h;
  const bool ok = tok < s.lq && pk.ok;
  const uint4* src = reinterpret_cast<const uint4*>(P.q + (P.packed ? 0 : s.b * P.q_b) + (int64_t)(s.q_start + tok) * P.q_t + h * P.q_h);
  uint32_t top = 0u;
#pragma unroll 4
  for (int e = 0; e < 16; ++e) {
    const uint4 x = ok ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
    top = __vmaxu2(top, x.x & 0x7fff7fffu);
    top = __vmaxu2(top, x.y & 0x7fff7fffu);
    top = __vmaxu2(top, x.z & 0x7fff7fffu);
    top = __vmaxu2(top, x.w & 0x7fff7fffu);
  }
  top = max(top & 0xffffu, top >> 16);
  // Exponent of s, so that amax / s is in (224, 448]. A row with infinities or
  // NaN has them as e4m3 NaN: its scores are NaN, as the formula's are.
  const bool finite = top < 0x7f80u;
  const int e2 = finite && top ? max(-126, (int)(top >> 7) - 127 - 8 + ((top & 0x7fu) > 96u ? 1 : 0)) : 0;
  const float inv = finite ? __uint_as_float((uint32_t)(127 - e2) << 23) : __uint_as_float(0x7fc00000u);
  reinterpret_cast<float*>(c.smem + T::OFF_QS)[kBlockM * i + r] = __uint_as_float((uint32_t)(127 + e2) << 23);
  const uint32_t dst = c.sbase + T::OFF_Q + i * T::Q_TILE_BYTES + r * 128;
#pragma unroll 1
  for (int e = 0; e < 8; ++e) {   // 16 depths at a time
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint4 x = ok ? __ldg(src + 2 * e + k) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float f[4], b[4];
        f[0] = __uint_as_float(w[2 * y] << 16) * inv;
        f[1] = __uint_as_float(w[2 * y] & 0xffff0000u) * inv;
        f[2] = __uint_as_float(w[2 * y + 1] << 16) * inv;
        f[3] = __uint_as_float(w[2 * y + 1] & 0xffff0000u) * inv;
        const uint32_t q1 = ptx::pack_e4m3x4(f[0], f[1], f[2], f[3]);
        ptx::e4m3x2_to_float2(q1 & 0xffffu, b[0], b[1]);
        ptx::e4m3x2_to_float2(q1 >> 16, b[2], b[3]);
        hi[2 * k + y] = q1;
        lo[2 * k + y] = ptx::pack_e4m3x4(f[0] - b[0], f[1] - b[1], f[2] - b[2], f[3] - b[3]);
      }
    }
    const uint32_t at = dst + ((e ^ (r & 7)) << 4);
    ptx::st_shared_v4(at, hi[0], hi[1], hi[2], hi[3]);
    ptx::st_shared_v4(at + T::CHUNK_BYTES, lo[0], lo[1], lo[2], lo[3]);
  }
  ptx::fence_async_shared();   // before the MMAs read the tiles
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(c.bar(BAR_Q_FULL + i));
}

template <class T, int CAUSAL>
__device__ void role_correction(const Tc05Params& P, const Ctx& c) {
  const int tid = threadIdx.x - 256;
  const uint32_t lane_base = (uint32_t)(((threadIdx.x >> 5) & 3) * 32) << 16;
  const float* rcpl_sm = reinterpret_cast<const float*>(c.smem + T::OFF_RCPL);
  [[maybe_unused]] const PackedRow pk(P, tid);
  Ring<2> sched;
  uint32_t stats_phase[2] = {0, 0}, ofinal_phase[2] = {0, 0};
  [[maybe_unused]] Widen<T> widen;
  [[maybe_unused]] uint32_t q_empty_phase = 0;   // QSPLIT
  while (true) {
    if (!wait_warp(c, BAR_SCHED_FULL + sched.idx, sched.phase, kRoleCorrection)) return;
    const SchedSlot s = read_slot<CAUSAL, T::PAGED>(c, sched.idx, T::OFF_SCHED);
    ptx::mbar_arrive(c.bar(BAR_SCHED_EMPTY + sched.idx));
    sched.next();
    if (!s.valid) return;
    const Geo g = tile_geo<T, CAUSAL>(s, c.rank, P.pack_tokens);
    if constexpr (T::C8) {
      if (g.n[1] > 0) {
        widen.begin(P, c, s, g.n[1]);
        if constexpr (T::QSPLIT) {
          if (!wait_warp(c, BAR_Q_EMPTY, q_empty_phase ^ 1u, kRoleCorrection)) { ptx::cp_async_wait<0>(); return; }
          split_q<T>(P, c, s, g.row[0], 0);
          if (!wait_warp(c, BAR_Q_EMPTY1, q_empty_phase ^ 1u, kRoleCorrection)) { ptx::cp_async_wait<0>(); return; }
          split_q<T>(P, c, s, g.row[1], 1);
          q_empty_phase ^= 1u;
        }
        if (!widen.run(P, c, s, g.n[1])) return;
      }
    }
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      // Epilogue of Q tile i: O = O / l, rounded once to bf16, stored row by row.
      if (!wait_warp(c, BAR_STATS + i, stats_phase[i], kRoleCorrection)) return;
      stats_phase[i] ^= 1u;
      const float rl = rcpl_sm[i * kBlockM + tid];
      ptx::mbar_arrive(c.bar(BAR_STATS_FREE + i));
      const int qi = T::PAGED ? g.row[i] + pk.tok : g.row[i] + tid;
      const int h = T::PAGED ? s.h * P.pack + pk.h : s.h;
      const bool row_valid = qi < s.lq && (!T::PAGED || pk.ok);
      const bool partial = T::PAGED ? listed<CAUSAL>() && s.split >= 0 : splits_keys<CAUSAL>(P);
      const int64_t part_at = T::PAGED ? (int64_t)s.split * kRowsPerTile + kBlockM * i + tid : partial_row(P, s, qi);
      uint16_t* orow = P.o + (int64_t)s.b * P.o_stride_b + (int64_t)(s.q_start + qi) * P.o_stride_t +
                       (int64_t)h * P.o_stride_h;
      if (g.n[i] > 0) {
        if (!wait_warp(c, BAR_O_FINAL + i, ofinal_phase[i], kRoleCorrection)) return;
        ofinal_phase[i] ^= 1u;
        ptx::tc_fence_after();
        const uint32_t tO = c.tmem + lane_base + T::tm_o(i);
        if (partial) {
          // Split-KV range: normalised partial O in fp32 for the merge.
          float* prow = P.o_part + part_at * T::DV;
#pragma unroll 1
          for (int q = 0; q < T::DV / 32; ++q) {
            uint32_t r[32];
            ptx::tmem_ld32(tO + 32 * q, r);
            ptx::tmem_wait_ld();
            if (row_valid) store_row_chunk_f32(prow + 32 * q, r, rl);
          }
        } else {
#pragma unroll
          for (int q = 0; q < T::DV / 32; ++q) {
            uint32_t r[32];
            ptx::tmem_ld32(tO + 32 * q, r);
            ptx::tmem_wait_ld();
            if (row_valid) store_row_chunk<T>(orow + 32 * q, r, rl, P.o_store32 != 0);
          }
        }
      } else if (row_valid && partial) {
        // An empty key range (a short packed sequence, or under the causal
        // mask a range this tile's rows do not reach): a zero partial row
        // (its LSE is -inf, so the merge gives it no weight).
        float4* d = reinterpret_cast<float4*>(P.o_part + part_at * T::DV);
#pragma unroll 1
        for (int e = 0; e < T::DV / 4; ++e) d[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (row_valid) {
        uint4* d = reinterpret_cast<uint4*>(orow);
#pragma unroll
        for (int e = 0; e < T::DV / 8; ++e) d[e] = make_uint4(0u, 0u, 0u, 0u);
      }
      ptx::tc_fence_before();
      if constexpr (T::PAIR) {
        // one arrival per warp on the first CTA's barrier (its MMAs write both CTAs' O)
        __syncwarp();
        if ((threadIdx.x & 31) == 0) arrive_lead(c, BAR_O_FREE + i);
      } else {
        ptx::mbar_arrive(c.bar(BAR_O_FREE + i));
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
template <int N>
__device__ __forceinline__ void setmaxnreg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void setmaxnreg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

template <class T, int CAUSAL>
__global__ void __launch_bounds__(512, 1) fa_tc05_kernel(const __grid_constant__ Tc05Params P) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctx c;
  c.smem = smem;
  c.sbase = ptx::smem_u32(smem);
  c.ws = P.ws;
  c.abort_flag = reinterpret_cast<volatile int*>(smem + T::OFF_ABORT);
  c.bar_off = T::OFF_BAR;
  c.timeout_ns = P.timeout_ns;
  c.rank = T::PAIR ? ptx::cluster_ctarank() : 0u;
  c.peer_abort = 0u;
  if (c.sbase & 1023u) {  // the swizzled tiles need a 1024-byte aligned base (same in both CTAs of a pair)
    if constexpr (!T::FP8) ptx::grid_dependency_wait();
    if (threadIdx.x == 0) atomicCAS(&P.ws[kWsErrorCode], 0u, 2u);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Barriers that the second CTA of a pair reports to per warp (4 warps per CTA).
  const uint32_t warp_count = T::PAIR ? 8u : 128u;
  if (threadIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(c.bar(BAR_Q_FULL + i), T::Q_FILL);
      ptx::mbar_init(c.bar(BAR_S_FULL + i), 1);
      ptx::mbar_init(c.bar(BAR_P_LO + i), warp_count);
      ptx::mbar_init(c.bar(BAR_STATS + i), 128);
      ptx::mbar_init(c.bar(BAR_P_HI + i), warp_count);
      ptx::mbar_init(c.bar(BAR_ORDER + i), 1);
      ptx::mbar_init(c.bar(BAR_O_FINAL + i), 1);
      ptx::mbar_init(c.bar(BAR_O_FREE + i), warp_count);
      ptx::mbar_init(c.bar(BAR_STATS_FREE + i), 128);
      ptx::mbar_init(c.bar(BAR_KS + i), 128);
      ptx::mbar_init(c.bar(BAR_SCHED_FULL + i), 1);
      // a pair's second CTA runs no MMA issuers, an e4m3 cache no V producer warp
      ptx::mbar_init(c.bar(BAR_SCHED_EMPTY + i), kSchedConsumers - (c.rank != 0 ? 2u : 0u) - (T::C8 ? 1u : 0u));
      ptx::mbar_init(c.bar(BAR_WORK_FULL + i), 1);
      ptx::mbar_init(c.bar(BAR_WORK_EMPTY + i), 1);
      ptx::mbar_init(c.bar(BAR_SM_TURN + i), 128);
    }
    ptx::mbar_init(c.bar(BAR_Q_EMPTY), 1);
    ptx::mbar_init(c.bar(BAR_Q_EMPTY1), 1);
    ptx::mbar_init(c.bar(BAR_DRAIN), 2);
#pragma unroll
    for (int s = 0; s < T::NK; ++s) {
      ptx::mbar_init(c.bar(T::BAR_K_FULL + s), T::K_FILL);
      ptx::mbar_init(c.bar(T::BAR_K_EMPTY + s), 2);
    }
#pragma unroll
    for (int s = 0; s < T::NV; ++s) {
      ptx::mbar_init(c.bar(T::BAR_V_FULL + s), T::V_FILL);
      ptx::mbar_init(c.bar(T::BAR_V_EMPTY + s), 2);
    }
    if constexpr (T::QSPLIT) {
#pragma unroll
      for (int s = 0; s < kScaleSlots; ++s) ptx::mbar_init(c.bar(T::BAR_SCALES + s), 1);
    } else if constexpr (T::PAGED) {
      ptx::mbar_init(c.bar(T::BAR_V_TAIL), 1);
    }
    *c.abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    if constexpr (T::PAIR) {
      ptx::tmem_alloc_pair(c.sbase + T::OFF_TMEM_SLOT, T::TMEM_COLS);
      ptx::tmem_relinquish_pair();
    } else {
      ptx::tmem_alloc(c.sbase + T::OFF_TMEM_SLOT, T::TMEM_COLS);
      ptx::tmem_relinquish();
    }
  }
  if (warp == 14 && lane == 0) {
    if constexpr (!T::QSPLIT) ptx::prefetch_tmap(&P.tm_q);
    if constexpr (!T::C8 || T::QSPLIT) ptx::prefetch_tmap(&P.tm_k);
    if constexpr (!T::C8) ptx::prefetch_tmap(&P.tm_v);
    if (T::DR > 0) {
      ptx::prefetch_tmap(&P.tm_qr);
      ptx::prefetch_tmap(&P.tm_kr);
    }
  }
  ptx::tc_fence_before();
  // A pair's barriers must be initialised in both CTAs before either CTA
  // copies into, or arrives on, the other's.
  __syncwarp();
  if constexpr (T::PAIR) ptx::cluster_sync();
  else __syncthreads();
  ptx::tc_fence_after();
  c.tmem = *reinterpret_cast<volatile uint32_t*>(smem + T::OFF_TMEM_SLOT);
  if constexpr (T::PAIR) c.peer_abort = ptx::mapa(c.sbase + T::OFF_ABORT, c.rank ^ 1u);
  // The set-up above touches no global memory, so it may overlap the
  // previous kernel on the stream (programmatic dependent launch); from here
  // on the kernel reads inputs and writes outputs and the workspace, so it
  // waits until that kernel has completed and its writes are visible. (The
  // FP8 variants are never launched that way: any added code in them
  // measured ~1 % slower, their softmax being at its register ceiling.)
  if constexpr (!T::FP8) ptx::grid_dependency_wait();   // returns at once without a dependency

  const int wg = warp >> 2;
  if (wg < 2) {
    setmaxnreg_inc<T::REG_SOFTMAX>();
    role_softmax<T, CAUSAL>(P, c, wg);
  } else if (wg == 2) {
    setmaxnreg_dec<T::REG_CORR>();
    role_correction<T, CAUSAL>(P, c);
  } else {
    setmaxnreg_dec<T::REG_MISC>();
    if (warp == 12 || warp == 13) {
      if (lane == 0 && c.rank == 0) role_mma<T, CAUSAL>(P, c, warp - 12);
      __syncwarp();
    }
    else if (warp == 14) role_load_qk<T, CAUSAL>(P, c);
    else if constexpr (!T::C8) role_load_v<T, CAUSAL>(P, c);
  }

  ptx::tc_fence_before();
  // Both CTAs of a pair are done with the MMAs (which use both CTAs' tensor
  // and shared memory) before either frees its tensor memory or exits.
  __syncwarp();
  if constexpr (T::PAIR) ptx::cluster_sync();
  else __syncthreads();
  if (warp == 12) {
    ptx::tc_fence_after();
    if constexpr (T::PAIR) ptx::tmem_dealloc_pair(c.tmem, T::TMEM_COLS);
    else ptx::tmem_dealloc(c.tmem, T::TMEM_COLS);
  }
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&P.ws[kWsDoneCounter], 1u) == gridDim.x - 1) {
      atomicExch(&P.ws[kWsTileCounter], 0u);
      atomicExch(&P.ws[kWsDoneCounter], 0u);
      __threadfence();
    }
  }
}

// Launch configuration of a pair variant: clusters of two CTAs.
template <class T>
cudaLaunchConfig_t pair_config(int grid, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid, 1, 1);
  cfg.blockDim = dim3(512, 1, 1);
  cfg.dynamicSmemBytes = T::SMEM_BYTES;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <class T, int CAUSAL>
cudaError_t tc05_launch_tc(const Tc05Params& prm, int grid, cudaStream_t stream) {
  constexpr auto kern = fa_tc05_kernel<T, CAUSAL>;
  return launch_with_smem<kern>(T::SMEM_BYTES, [&]() -> cudaError_t {
    if constexpr (T::PAIR) {
      if (grid % 2 != 0) return cudaErrorInvalidValue;
      cudaLaunchAttribute attr[1];
      const cudaLaunchConfig_t cfg = pair_config<T>(grid, stream, attr);
      const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, prm);
      if (e != cudaSuccess) return e;
    } else if (T::FP8 || !prm.dependent_launch) {
      kern<<<grid, 512, T::SMEM_BYTES, stream>>>(prm);
    } else {
      // programmatic dependent launch: set-up overlaps the previous kernel's
      // last CTAs (the kernel waits before its first global access)
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
      attr[0].val.programmaticStreamSerializationAllowed = 1;
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3((unsigned)grid);
      cfg.blockDim = dim3(512);
      cfg.dynamicSmemBytes = T::SMEM_BYTES;
      cfg.stream = stream;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, prm);
      if (e != cudaSuccess) return e;
    }
    return cudaGetLastError();
  });
}

template <class T>
cudaError_t tc05_launch_t(int mask, const Tc05Params& prm, int grid, cudaStream_t stream) {
  if (mask == kMaskNone) return tc05_launch_tc<T, kMaskNone>(prm, grid, stream);
  if (mask == kMaskCausal) return tc05_launch_tc<T, kMaskCausal>(prm, grid, stream);
  if (mask == kMaskNoneSplit) return tc05_launch_tc<T, kMaskNoneSplit>(prm, grid, stream);
  if constexpr (!T::PAIR) {
    if (mask == kMaskCausalSplit) return tc05_launch_tc<T, kMaskCausalSplit>(prm, grid, stream);
  }
  return cudaErrorInvalidValue;
}

// Clusters of a pair variant that can be resident at once on the current
// device (0 if the query fails or the variant is not a pair variant).
template <class T>
int tc05_max_clusters_t() {
  if constexpr (!T::PAIR) {
    return 0;
  } else {
    auto kern = fa_tc05_kernel<T, kMaskCausal>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM_BYTES) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = pair_config<T>(2, nullptr, attr);
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return n;
  }
}

template <class T>
Tc05Config tc05_config_t() {
  Tc05Config c;
  c.smem_bytes = T::SMEM_BYTES;
  c.k_stages = T::NK;
  c.v_stages = T::NV;
  c.threads = 512;
  c.tmem_cols = (int)T::TMEM_COLS;
  return c;
}

using TraitsD64 = Tc05Traits<64, 0, 64, false>;
using TraitsD128 = Tc05Traits<128, 0, 128, false>;
using TraitsD128R64 = Tc05Traits<128, 64, 128, false>;
using TraitsFp8D128 = Tc05Traits<128, 0, 128, true>;
using TraitsFp8QkvD128 = Tc05Traits<128, 0, 128, true, true>;
using TraitsD128Pair = Tc05Traits<128, 0, 128, false, false, true>;
using TraitsD128R64Pair = Tc05Traits<128, 64, 128, false, false, true>;
using TraitsPagedD64 = Tc05Traits<64, 0, 64, false, false, false, true>;
using TraitsPagedD128 = Tc05Traits<128, 0, 128, false, false, false, true>;
using TraitsPaged8D64 = Tc05Traits<64, 0, 64, false, false, false, true, true>;
using TraitsPaged8D128 = Tc05Traits<128, 0, 128, false, false, false, true, true>;

cudaError_t tc05_launch_d64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_d128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_d128r64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_fp8d128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_fp8qkvd128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_d128pair(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_d128r64pair(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_pagedd64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_pagedd128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_paged8d64(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
cudaError_t tc05_launch_paged8d128(int mask, const Tc05Params& prm, int grid, cudaStream_t stream);
int tc05_max_clusters_d128pair();
int tc05_max_clusters_d128r64pair();

}  // namespace af
