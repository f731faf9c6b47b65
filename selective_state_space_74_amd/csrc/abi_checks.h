// Host-side checks shared by the ABI sources: byte spans of strided tensors,
// overlap and alignment.  Pure host code (no HIP call).
#pragma once

#include <stdint.h>

#include <numeric>

#include "ssm.h"

namespace ssm {

struct Span {  // byte range [lo, hi)
  uintptr_t lo = 0, hi = 0;
  bool empty() const { return hi <= lo; }
};

inline bool overlap(const Span& a, const Span& b) {
  return !a.empty() && !b.empty() && a.lo < b.hi && b.lo < a.hi;
}

// Bytes touched by a (n0, n1, n2) tensor with strides (s0, s1, 1).
inline Span span3(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2,
           int64_t esz) {
  Span s;
  if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0) return s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>(((n0 - 1) * s0 + (n1 - 1) * s1 + n2) * esz);
  return s;
}

inline Span span1(const void* p, int64_t n, int64_t esz) { return span3(p, 1, 0, 1, 0, n, esz); }

// Bytes touched by a (n0, n1, n2, n3) tensor with strides (s0, s1, s2, 1).
inline Span span4(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2,
           int64_t s2, int64_t n3, int64_t esz) {
  Span s;
  if (!p || n0 <= 0 || n1 <= 0 || n2 <= 0 || n3 <= 0) return s;
  s.lo = reinterpret_cast<uintptr_t>(p);
  s.hi = s.lo + static_cast<uintptr_t>(((n0 - 1) * s0 + (n1 - 1) * s1 + (n2 - 1) * s2 + n3) * esz);
  return s;
}

// A (n0, n1, n2) tensor with strides (s0, s1, 1), as rows of n2 elements.
struct Rows {
  Span span;
  int64_t s0 = 0, s1 = 0, row = 0;  // bytes
};

inline Rows rows3(const void* p, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2,
                  int64_t esz) {
  return Rows{span3(p, n0, s0, n1, s1, n2, esz), n0 > 1 ? s0 * esz : 0, n1 > 1 ? s1 * esz : 0, n2 * esz};
}

// Whether two such tensors share bytes.  Slices of one wider tensor (the same
// strides, in either order) interleave without sharing any: every row of a tensor
// begins at the same place of a period that both strides are multiples of.
inline bool overlap(const Rows& a, const Rows& b) {
  if (!overlap(a.span, b.span)) return false;
  const int64_t period = std::gcd(a.s0, a.s1);
  if (a.s0 != b.s0 || a.s1 != b.s1 || period == 0) return true;
  const Rows& lo = a.span.lo <= b.span.lo ? a : b;
  const Rows& hi = a.span.lo <= b.span.lo ? b : a;
  const int64_t off = static_cast<int64_t>((hi.span.lo - lo.span.lo) % static_cast<uintptr_t>(period));
  return off < lo.row || off + hi.row > period;
}
inline bool overlap(const Rows& a, const Span& b) { return overlap(a.span, b); }

// Whether two rows of one output can share bytes.
inline bool rows_collide(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2) {
  return (n1 > 1 && s1 < n2) || (n0 > 1 && s0 < (n1 > 0 ? (n1 - 1) * s1 : 0) + n2);
}

// B/C groups: 0 or 1 is one group; otherwise it must divide dim.
inline int64_t groups_of(int64_t ngroups) { return ngroups > 1 ? ngroups : 1; }
inline bool bad_groups(int64_t ngroups, int64_t dim) {
  return ngroups < 0 || (dim > 0 && dim % groups_of(ngroups) != 0);
}

inline bool misaligned(const void* p, int64_t align) {
  return p && (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align)) != 0;
}

inline int64_t io_size(int32_t dt) { return dt == SSM_BF16 ? 2 : 4; }

// Token indices are 32-bit inside the scan kernel.
constexpr int64_t kMaxSeqlen = (int64_t{1} << 31) - 64;
constexpr int64_t kCkptTokens = SSM_CHECKPOINT_TOKENS;

}  // namespace ssm
