// Checks of matrices that need only their elements' alignment, and the memory
// that they span (host only).
#pragma once
#include <stdint.h>

#include <vector>

#include "../../include/muon.h"
#include "muon_span.h"

namespace muon {

constexpr int64_t kMaxRows = int64_t(1) << 30;
// Elements from a matrix's first to its last: more than any memory, and bytes and
// multiples of it stay far below 2^63.
constexpr int64_t kMaxSpan = int64_t(1) << 52;

inline int esize(int dt) { return dt == MUON_BF16 ? 2 : 4; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Whether n pieces of `width` elements, `pitch` apart, are within kMaxSpan.
inline bool fits(int64_t n, int64_t pitch, int64_t width) {
  return width <= kMaxSpan && (n <= 1 || n - 1 <= (kMaxSpan - width) / pitch);
}

// A matrix of any size, zero included; rows need only element alignment.
inline int check_dense(const muon_mat& m) {
  if (m.dtype != MUON_BF16 && m.dtype != MUON_F32) return MUON_E_DTYPE;
  if (m.rows < 0 || m.cols < 0 || m.rows > kMaxRows || m.cols > kMaxRows) return MUON_E_SHAPE;
  if (m.rows == 0 || m.cols == 0) return MUON_OK;
  if (m.ld < m.cols || m.ld > (int64_t(1) << 40) || !fits(m.rows, m.ld, m.cols)) return MUON_E_SHAPE;
  if (!m.ptr) return MUON_E_NULL;
  if (reinterpret_cast<uintptr_t>(m.ptr) % esize(m.dtype)) return MUON_E_ALIGN;
  return MUON_OK;
}

inline void add_span(std::vector<Span>& v, const void* p, size_t bytes, bool write) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  if (p && bytes) v.push_back({a, a + bytes, bytes, bytes, write});
}

inline void add_span(std::vector<Span>& v, const muon_mat& m, bool write) {
  if (m.rows == 0 || m.cols == 0) return;
  const uintptr_t a = reinterpret_cast<uintptr_t>(m.ptr);
  const size_t es = esize(m.dtype);
  v.push_back({a, a + (size_t(m.rows - 1) * m.ld + m.cols) * es, size_t(m.ld) * es,
               size_t(m.cols) * es, write});
}

}  // namespace muon
