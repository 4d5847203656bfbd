// Whether two matrices in memory share a byte (host only).  Exact, so that slices of one wider
// matrix beside each other are told from slices that overlap.
#pragma once

#include <stdint.h>

#include <utility>

namespace gc {

// rows pieces of `width` bytes, `stride` >= width bytes apart; nothing where at, width or rows is 0.
struct Area {
  uintptr_t at;
  int64_t width, stride, rows;
  uintptr_t end() const { return at + (uintptr_t)((rows - 1) * stride + width); }
};

// Whether the piece [lo, hi) meets a row of m: the first row that ends past lo has to start before hi.
inline bool meets(uintptr_t lo, uintptr_t hi, const Area& m) {
  int64_t r = 0;
  if (lo >= m.at + (uintptr_t)m.width) r = (int64_t)((lo - m.at - (uintptr_t)m.width) / (uintptr_t)m.stride) + 1;
  return r < m.rows && m.at + (uintptr_t)(r * m.stride) < hi;
}

inline bool overlap(Area a, Area b) {
  for (Area* m : {&a, &b}) {
    if (m->at == 0 || m->width == 0 || m->rows == 0) return false;
    if (m->rows == 1 || m->stride == m->width) *m = {m->at, (m->rows - 1) * m->stride + m->width, (m->rows - 1) * m->stride + m->width, 1};
  }
  if (a.end() <= b.at || b.end() <= a.at) return false;
  if (b.at < a.at) std::swap(a, b);
  if (a.rows == 1) return meets(a.at, a.end(), b);
  if (b.rows == 1) return meets(b.at, b.end(), a);
  if (a.stride == b.stride) {
    // row j of b starts `phase` after the start of row first + j of a
    const int64_t d = (int64_t)(b.at - a.at), first = d / a.stride, phase = d - first * a.stride;
    return (phase < a.width && first < a.rows) || (phase + b.width > a.stride && first + 1 < a.rows);
  }
  if (a.rows > b.rows) std::swap(a, b);
  for (int64_t r = 0; r < a.rows; ++r) {     // different strides: row by row; rows that do overlap end it soon
    const uintptr_t lo = a.at + (uintptr_t)(r * a.stride);
    if (meets(lo, lo + (uintptr_t)a.width, b)) return true;
  }
  return false;
}

}  // namespace gc
