// Whether rows that a call writes lie where it reads or writes others.
#pragma once
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

namespace af {

// Rows [n0][n1][n2] of `bytes` bytes each, strides in bytes (of no meaning where n is 1).
struct RowsAt {
  uintptr_t p;
  int64_t n[3], s[3];
  int64_t bytes;
  RowsAt(const void* base, int64_t n0, int64_t n1, int64_t n2, const int64_t* stride, int64_t dim)
      : p(reinterpret_cast<uintptr_t>(base)), n{n0, n1, n2}, s{2 * stride[0], 2 * stride[1], 2 * stride[2]}, bytes(2 * dim) {}
  uintptr_t end() const {
    uintptr_t e = p + static_cast<uintptr_t>(bytes);
    for (int i = 0; i < 3; ++i) e += static_cast<uintptr_t>((n[i] - 1) * s[i] * (n[i] > 1));
    return e;
  }
};

// Where rows of one stride each may be: apart (for sure), the same rows, or meeting.
// Strides that differ cannot be told apart once the ranges of addresses meet: unsure.
enum class Overlap { kApart, kSame, kMeet, kUnsure };

// Whether some d + sum x[i] s[i] with x[i] in lo[i] .. hi[i] is smaller than `bytes`, the
// strides in descending order: the two multiples on either side of d are tried, which finds
// it where a stride is at least as long as what lies inside.
inline bool reaches(int64_t d, const int64_t* s, const int64_t* lo, const int64_t* hi, int dims, int64_t bytes) {
  if (dims == 0) return d < bytes && -d < bytes;
  if (s[0] == 0) return reaches(d, s + 1, lo + 1, hi + 1, dims - 1, bytes);
  const int64_t down = -d / s[0] - ((-d) % s[0] < 0 ? 1 : 0);
  for (int64_t x : {down, down + 1})
    if (reaches(d + std::min(std::max(x, lo[0]), hi[0]) * s[0], s + 1, lo + 1, hi + 1, dims - 1, bytes)) return true;
  return false;
}

inline Overlap overlap(const RowsAt& a, const RowsAt& b) {
  for (int i = 0; i < 3; ++i)
    if (a.n[i] <= 0 || b.n[i] <= 0) return Overlap::kApart;
  if (a.p >= b.end() || b.p >= a.end()) return Overlap::kApart;
  int64_t s[3], lo[3], hi[3];
  bool same = a.p == b.p;
  for (int i = 0; i < 3; ++i) {
    if (a.n[i] > 1 && b.n[i] > 1 && a.s[i] != b.s[i]) return Overlap::kUnsure;
    same = same && a.n[i] == b.n[i];
    s[i] = a.n[i] > 1 ? a.s[i] : (b.n[i] > 1 ? b.s[i] : 0);
    lo[i] = 1 - b.n[i];
    hi[i] = a.n[i] - 1;
  }
  if (same) return Overlap::kSame;
  for (int i : {0, 1, 0})   // sorted
    if (s[i] < s[i + 1]) {
      std::swap(s[i], s[i + 1]);
      std::swap(lo[i], lo[i + 1]);
      std::swap(hi[i], hi[i + 1]);
    }
  return reaches(static_cast<int64_t>(a.p - b.p), s, lo, hi, 3, a.bytes) ? Overlap::kMeet : Overlap::kApart;
}

// What is wrong with rows `out` that are turned from `in` (in place, if they are the same)
// while `others` are read or written; NULL: nothing.
inline const char* misplaced(const RowsAt& out, const RowsAt& in, std::initializer_list<RowsAt> others) {
  if (out.n[0] <= 0 || out.n[1] <= 0 || out.n[2] <= 0) return nullptr;
  for (int i = 0; i < 3; ++i)
    if (out.n[i] > 1 && out.s[i] == 0) return "has rows in one place (a stride of 0)";
  const Overlap o = overlap(out, in);
  if (o == Overlap::kMeet || o == Overlap::kUnsure) return "shares memory with its input without being it";
  for (const RowsAt& x : others) {
    const Overlap y = overlap(out, x);
    if (y == Overlap::kMeet || y == Overlap::kSame) return "shares memory with other rows of the call";
  }
  return nullptr;
}

}  // namespace af
