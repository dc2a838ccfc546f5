// Argument checks shared by the C ABI's files: dtypes, alignment, and the
// address ranges a call reads and writes.
#pragma once

#include <cstddef>
#include <cstdint>

#include "fsdp_mi355x.h"

namespace fsdp {

inline bool valid_dtype(int32_t dt) { return dt == FSDP_F32 || dt == FSDP_BF16; }
inline int64_t dtype_size(int32_t dt) { return dt == FSDP_F32 ? 4 : 2; }

// Elements from the first of n rows, ld apart, to behind `cols` of the last one;
// -1 if that is no length an array can have.
inline int64_t reach(int64_t n, int64_t ld, int64_t cols) {
  if (n <= 0) return 0;
  const double far = static_cast<double>(n - 1) * static_cast<double>(ld) + static_cast<double>(cols);
  return far < 0x1p56 ? (n - 1) * ld + cols : -1;
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};
inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(const Range& a, const Range& b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}
// The address ranges one call reads or writes, kept inline: at most 64
// gradient replicas, receivers or arrays, plus the state arrays.  The
// argument checks allocate nothing.
struct Ranges {
  Range r[FSDP_MAX_RANKS + 8];
  int n = 0;
  void push_back(const Range& x) {
    if (n < FSDP_MAX_RANKS + 8) r[n++] = x;
  }
  const Range* begin() const { return r; }
  const Range* end() const { return r + n; }
  size_t size() const { return static_cast<size_t>(n); }
  const Range& operator[](size_t i) const { return r[i]; }
};

template <typename L>
bool any_overlap(const L& rs) {
  for (size_t i = 0; i < rs.size(); ++i)
    for (size_t j = i + 1; j < rs.size(); ++j)
      if (overlap(rs[i], rs[j])) return true;
  return false;
}

}  // namespace fsdp
