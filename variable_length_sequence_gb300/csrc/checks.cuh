// Host checks that the entry points share: alignment, element types, and which
// buffers of a call share bytes.
#pragma once

#include <stdint.h>

#include "nsp.h"

namespace nsp {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int32_t kMaxHeads = 1 << 15;           // keeps grids, coordinates and counts in range

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool dtype_ok(int32_t t) { return t == NSP_F32 || t == NSP_BF16; }
inline int64_t elem_bytes(int32_t t) { return t == NSP_BF16 ? 2 : 4; }

// rows of `row` bytes, `step` bytes apart
struct Span {
  uintptr_t base;
  int64_t rows, step, row;
  uintptr_t end() const { return base + (uintptr_t)((rows - 1) * step + row); }
};

// Whether two spans share a byte.  Spans of the same step (views of one
// tensor's columns) are compared column by column; others by their extents.
inline bool overlap(const Span& a, const Span& b) {
  if (a.rows < 1 || b.rows < 1 || a.row < 1 || b.row < 1) return false;
  if (a.end() <= b.base || b.end() <= a.base) return false;
  if (a.step != b.step || a.row > a.step || b.row > b.step) return true;
  const int64_t off = ((int64_t)(b.base - a.base) % a.step + a.step) % a.step;
  return off < a.row || off + b.row > a.step;
}

inline bool same_rows(const Span& a, const Span& b) {
  return a.base == b.base && a.rows == b.rows && a.step == b.step;
}

// `rows` rows of `row` bytes, one behind the other; none where p is NULL
inline Span packed(const void* p, int64_t rows, int64_t row) {
  return {reinterpret_cast<uintptr_t>(p), p ? rows : 0, row, row};
}

}  // namespace nsp
