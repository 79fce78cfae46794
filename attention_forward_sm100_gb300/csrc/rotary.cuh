// Rotation of 16-byte pieces (eight bf16) of a head by its token's position.
//
// A pair (x1, x2) becomes (x1 c - x2 s, x2 c + x1 s): two products, each
// rounded, and their sum, rounded; never contracted to a fused multiply-add, so
// that every kernel that rotates gives the same bits.
#pragma once
#include <stdint.h>

#include "ptx.cuh"

namespace af {

// cosines (or sines) of a position, from pair i0 on
template <int N>
__device__ __forceinline__ void load_angles(const float* row, int i0, float (&a)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
    a[i] = v.x;
    a[i + 1] = v.y;
    a[i + 2] = v.z;
    a[i + 3] = v.w;
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t two) { return __uint_as_float(two << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t two) { return __uint_as_float(two & 0xffff0000u); }

// own * c + other * s: the second of a pair; with -s the first (negating a
// product is exact).
__device__ __forceinline__ float turned(float own, float other, float c, float s) {
  return __fadd_rn(__fmul_rn(own, c), __fmul_rn(other, s));
}

// W values that lie together.
template <int W>
struct TurnWord;
template <>
struct TurnWord<8> {
  using type = uint4;
  __device__ static __forceinline__ uint4 load(const uint8_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }
};
template <>
struct TurnWord<1> {
  using type = uint16_t;
  __device__ static __forceinline__ uint16_t load(const uint8_t* p) { return *reinterpret_cast<const uint16_t*>(p); }
};

// Sums (differences) of packed products. The products are packed, two to an instruction,
// the sums are not: packed additions of packed products are contracted to fused ones,
// whatever rounding they ask for.
template <bool MINUS = false>
__device__ __forceinline__ void sum2(uint64_t a, uint64_t b, float& lo, float& hi) {
  float a0, a1, b0, b1;
  ptx::f2_unpack(a, a0, a1);
  ptx::f2_unpack(b, b0, b1);
  lo = MINUS ? __fsub_rn(a0, b0) : __fadd_rn(a0, b0);
  hi = MINUS ? __fsub_rn(a1, b1) : __fadd_rn(a1, b1);
}
// Two pairs at once, as bf16: (a c - b s, b c + a s) of packed values.
__device__ __forceinline__ void turned2(uint64_t a, uint64_t b, uint64_t c, uint64_t s, uint32_t& y1, uint32_t& y2) {
  float lo, hi;
  sum2<true>(ptx::f2_mul(a, c), ptx::f2_mul(b, s), lo, hi);
  y1 = ptx::pack_bf16(lo, hi);
  sum2(ptx::f2_mul(b, c), ptx::f2_mul(a, s), lo, hi);
  y2 = ptx::pack_bf16(lo, hi);
}
__device__ __forceinline__ uint64_t f2_of(uint32_t two) { return ptx::f2_pack(bf16_lo(two), bf16_hi(two)); }
// ---- Whole rows: kHeads heads of a token by one thread
//
// Every byte moves once each way, and a token's line of the table (4 R bytes, for all its
// heads) once from L2: HBM bounds it, once little else is done. A thread takes one item
// of a token, an item being what is turned together: 16 bytes and, in the half layout,
// the 16 bytes R / 2 behind them (or 16 bytes that are only copied). It keeps the item's
// cosines and sines and goes through up to four (eight) neighbouring heads, whose loads are
// all in flight, those of a thread's first item before anything is known about its token.
// Packed rows of 23700 tokens, 40 heads of 128, 64 values of each turned, take 74 us of a
// floor of 72. (Heads looked up one by one, values turned one by one, tokens found before
// the first load, 62 % of the threads busy: 139. Appends of 41690 tokens with 48 heads, by
// shuffles among a head's lanes: 303 of 152, by this 162.)
constexpr int turn_heads(bool apart) { return apart ? 4 : 8; }   // 128 bytes of a thread on their way

struct TurnShape {
  const float* table;
  int32_t rot, interleaved, inverse;
  int32_t items, slots;          // of a head; threads of an item of a token
  int32_t first, first_slots;    // heads of the first segment, and their threads
  int32_t group, group2;         // heads of a thread, in the first segment and in others
  int32_t turned;                // heads up to this one are turned, those behind copied
  int32_t twos;                  // 1: 16-byte pieces that are only copied go two by two
};
// Sizes of a launch: heads[] of the segments that follow one another, the first `turned`
// of them turned.
inline TurnShape turn_shape(const float* table, int dim, int rot, bool interleaved, bool inverse, const int (&heads)[3],
                            int turned) {
  TurnShape t = {};
  const bool wide = rot % (interleaved ? 8 : 16) == 0;
  const int w = wide ? 8 : 1;
  t.table = table;
  t.rot = rot;
  t.interleaved = interleaved ? 1 : 0;
  t.inverse = inverse ? 1 : 0;
  // (two by two where their number is even: threads of such pieces alone keep half as much
  // on its way; 41690 tokens, 40 heads of 128, 64 of them turned, 183 us, with
  // this 140)
  const int pairs = rot / 2 / w, rest = dim / w - 2 * pairs;
  t.twos = wide && !interleaved && rest % 2 == 0 ? 1 : 0;
  t.items = wide && interleaved ? dim / w : pairs + (t.twos ? rest / 2 : rest);
  // (of each segment's own: with one for all, 88000 tokens with 32 heads of q and 2 of K and
  // of V, 64 depths, of which 16 turned, took 191 us of a floor of 120, with these 126)
  t.group = t.group2 = turn_heads(!(wide && interleaved));
  while (heads[0] % t.group) t.group /= 2;
  while (heads[1] % t.group2 || heads[2] % t.group2) t.group2 /= 2;
  t.first = heads[0];
  t.first_slots = heads[0] / t.group;
  t.slots = t.first_slots + (heads[1] + heads[2]) / t.group2;
  for (int i = 0; i < turned; ++i) t.turned += heads[i];
  return t;
}
inline bool turn_wide(const TurnShape& t) { return t.rot % (t.interleaved ? 8 : 16) == 0; }
// Pieces of eight of the interleaved layout hold both values of their pairs; else pairs
// are apart.
inline bool turn_apart(const TurnShape& t) { return !(turn_wide(t) && t.interleaved); }

// The head that a thread starts with: where it comes from and goes to, and the way to
// the next.
struct TurnHead {
  const uint8_t* src;
  int64_t src_next;
  uint8_t* dst;
  int64_t dst_next;
};

// Turns the rows of a block's tokens. source(token, h, head) fills the first half of
// `head`; prepare() has the block's threads find the tokens and ends with a barrier;
// after it, target(token, h, head) fills the second half and returns the token's line of
// the table, or -1 if it is not written. W values are handled at a time, 8 or 1; APART as
// turn_apart().
template <int W, bool APART, int THREADS, class Source, class Prepare, class Target>
__device__ __forceinline__ void turn_rows(const TurnShape& T, int tokens, Source source, Prepare prepare, Target target) {
  const int per_token = T.items * T.slots, total = tokens * per_token;
  static_assert(APART || W == 8, "");
  constexpr int HEADS = turn_heads(APART);
  const int half = APART ? T.rot / 2 / W : 0;   // the first items have two parts
  struct Unit {
    int token, h, heads, item, d, d2;
    bool pair, two;   // to be turned, with another part
  };
  auto unit_at = [&](int x) {
    Unit u;
    u.token = x / per_token;
    const int rest = x - u.token * per_token, slot = rest / T.items;
    u.item = rest - slot * T.items;
    const bool first = slot < T.first_slots;
    u.heads = first ? T.group : T.group2;
    u.h = first ? slot * T.group : T.first + (slot - T.first_slots) * T.group2;
    u.pair = u.item < half;
    // first value of the item, and of its other part
    u.two = APART && (u.pair || T.twos);
    u.d = (u.pair || !APART ? u.item : (T.twos ? 2 * u.item : u.item + half)) * W;
    u.d2 = u.d + (u.pair ? T.rot / 2 : W);
    if (W == 1 && u.pair && T.interleaved) {
      u.d = 2 * u.item;
      u.d2 = u.d + 1;
    }
    return u;
  };
  using Word = typename TurnWord<W>::type;
  Word a[HEADS], b[APART ? HEADS : 1];
  auto load = [&](const Unit& u) {
    TurnHead head;
    source(u.token, u.h, head);
#pragma unroll
    for (int y = 0; y < HEADS; ++y) {
      if (y < u.heads) {
        a[y] = TurnWord<W>::load(head.src + 2 * u.d);
        if (APART && u.two) b[y % (APART ? HEADS : 1)] = TurnWord<W>::load(head.src + 2 * u.d2);
        head.src += head.src_next;
      }
    }
  };
  int x = threadIdx.x;
  Unit u = unit_at(x);
  if (x < total) load(u);
  prepare();
#pragma unroll 1
  while (x < total) {
    TurnHead head;
    const int at = target(u.token, u.h, head);
    if (at >= 0) {
      const float* row = T.table + (int64_t)at * T.rot;
      const bool turn = u.h < T.turned;
      if constexpr (W == 8 && APART) {
        if (u.pair && turn) {
          float c[8], s[8];
          load_angles<8>(row, u.d, c);
          load_angles<8>(row, T.rot / 2 + u.d, s);
          uint64_t c2[4], s2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float s0 = T.inverse ? -s[2 * i] : s[2 * i], s1 = T.inverse ? -s[2 * i + 1] : s[2 * i + 1];
            c2[i] = ptx::f2_pack(c[2 * i], c[2 * i + 1]);
            s2[i] = ptx::f2_pack(s0, s1);
          }
#pragma unroll
          for (int y = 0; y < HEADS; ++y) {
            if (y < u.heads) {
              uint32_t p[4] = {a[y].x, a[y].y, a[y].z, a[y].w}, q[4] = {b[y].x, b[y].y, b[y].z, b[y].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) turned2(f2_of(p[i]), f2_of(q[i]), c2[i], s2[i], p[i], q[i]);
              a[y] = make_uint4(p[0], p[1], p[2], p[3]);
              b[y] = make_uint4(q[0], q[1], q[2], q[3]);
            }
          }
        }
      } else if constexpr (W == 8) {
        if (turn && u.d < T.rot) {
          float c[4], s[4];
          load_angles<4>(row, u.d / 2, c);
          load_angles<4>(row, T.rot / 2 + u.d / 2, s);
          uint64_t c2[4], s2[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float n = T.inverse ? -s[i] : s[i];
            c2[i] = ptx::f2_pack(c[i], c[i]);
            s2[i] = ptx::f2_pack(-n, n);
          }
#pragma unroll
          for (int y = 0; y < HEADS; ++y) {
            if (y < u.heads) {
              uint32_t p[4] = {a[y].x, a[y].y, a[y].z, a[y].w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {   // (x1, x2) (c, c) + (x2, x1) (-s, s)
                const float lo = bf16_lo(p[i]), hi = bf16_hi(p[i]);
                float y1, y2;
                sum2(ptx::f2_mul(ptx::f2_pack(lo, hi), c2[i]), ptx::f2_mul(ptx::f2_pack(hi, lo), s2[i]), y1, y2);
                p[i] = ptx::pack_bf16(y1, y2);
              }
              a[y] = make_uint4(p[0], p[1], p[2], p[3]);
            }
          }
        }
      } else {
        if (u.pair && turn) {
          const float c = __ldg(row + u.item), s0 = __ldg(row + T.rot / 2 + u.item), s = T.inverse ? -s0 : s0;
#pragma unroll
          for (int y = 0; y < HEADS; ++y) {
            if (y < u.heads) {
              const float p = __uint_as_float((uint32_t)a[y] << 16), q = __uint_as_float((uint32_t)b[y] << 16);
              a[y] = (uint16_t)ptx::pack_bf16(turned(p, q, c, -s), 0.f);
              b[y] = (uint16_t)ptx::pack_bf16(turned(q, p, c, s), 0.f);
            }
          }
        }
      }
#pragma unroll
      for (int y = 0; y < HEADS; ++y) {
        if (y < u.heads) {
          *reinterpret_cast<Word*>(head.dst + 2 * u.d) = a[y];
          if (APART && u.two) *reinterpret_cast<Word*>(head.dst + 2 * u.d2) = b[y % (APART ? HEADS : 1)];
          head.dst += head.dst_next;
        }
      }
    }
    x += THREADS;
    if (x < total) {
      u = unit_at(x);
      load(u);
    }
  }
}
// Tokens of a block: where there are many, the number that keeps most of its threads
// busy, as long as two rounds of eight blocks per SM are left.
inline int turn_tokens(const TurnShape& t, int64_t tokens, int threads, int most, int sms) {
  const int64_t per_token = (int64_t)t.items * t.slots, enough = tokens / (16ll * sms);
  int best = 1;
  double busy = 0;
  for (int n = 1; n <= most && n <= (enough < 1 ? 1 : enough) && (n == 1 || n * per_token <= 8ll * threads); ++n) {
    const int64_t units = n * per_token, rounds = (units + threads - 1) / threads;
    const double now = (double)units / (double)(rounds * threads);
    if (now > busy + 0.01) {
      busy = now;
      best = n;
    }
  }
  return best;
}

// Rotates the sixteen values (two pieces of eight) that each of the L lanes of a
// vector holds; `x` their bf16 bits, `row` the position's line of the table, of
// `rot` values (a multiple of 16). All lanes of the warp call it; where `on` is
// false the values are only widened.
template <int L>
__device__ __forceinline__ void rotate_lanes(const uint32_t (&x)[8], float (&f)[16], const float* row, int rot,
                                             bool interleaved, bool on) {
  const int lane = threadIdx.x % L;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    f[2 * i] = bf16_lo(x[i]);
    f[2 * i + 1] = bf16_hi(x[i]);
  }
  if (interleaved) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int p = 2 * lane + s;
      if (on && 8 * p < rot) {
        float c[4], n[4];
        load_angles<4>(row, 4 * p, c);
        load_angles<4>(row, rot / 2 + 4 * p, n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = f[8 * s + 2 * i], b = f[8 * s + 2 * i + 1];
          f[8 * s + 2 * i] = turned(a, b, c[i], -n[i]);
          f[8 * s + 2 * i + 1] = turned(b, a, c[i], n[i]);
        }
      }
    }
  } else {
    // the other of piece p's pairs is piece p + half or p - half, in another lane or in this one
    const int half = rot / 16;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int p = 2 * lane + s;
      const bool first = p < half;
      const int q = first ? p + half : (p < 2 * half ? p - half : p);
      uint32_t y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t mine = x[4 * ((half & 1) ? s ^ 1 : s) + i];   // (half odd: the other's piece is in the other slot)
        y[i] = __shfl_sync(0xffffffffu, mine, q / 2, L);
      }
      if (on && p < 2 * half) {
        float c[8], n[8];
        load_angles<8>(row, 8 * (first ? p : p - half), c);
        load_angles<8>(row, rot / 2 + 8 * (first ? p : p - half), n);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float o = (i & 1) ? bf16_hi(y[i / 2]) : bf16_lo(y[i / 2]);
          f[8 * s + i] = turned(f[8 * s + i], o, c[i], first ? -n[i] : n[i]);
        }
      }
    }
  }
}

}  // namespace af
