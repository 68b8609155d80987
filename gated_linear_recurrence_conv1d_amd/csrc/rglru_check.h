// rglru_check.h -- argument checks shared by the C ABI files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rglru.h"

namespace rglru {

inline size_t align_up(size_t v) {
  constexpr size_t kAlign = 256;  // workspace carve alignment
  return (v + kAlign - 1) / kAlign * kAlign;
}

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}

inline size_t elem_bytes(rglru_dtype dt) { return dt == RGLRU_BF16 ? 2 : 4; }

inline rglru_status hip_status(hipError_t e) { return e == hipSuccess ? RGLRU_OK : RGLRU_ERR_HIP; }

// `rows` runs of `width` bytes, `stride` bytes apart.
struct Rows {
  const void *p;
  size_t rows, width, stride;
  size_t span() const { return p && rows ? (rows - 1) * stride + width : 0; }
};

// Whether two sets of runs share a byte; sets of one stride may interleave (parts of the columns
// of one tensor), sets of different strides count as overlapping if their spans do.
inline bool overlaps(const Rows &a, const Rows &b) {
  if (!overlaps(a.p, a.span(), b.p, b.span())) return false;
  if (a.stride != b.stride || a.stride == 0) return true;
  const size_t s = a.stride;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  const size_t d = b0 >= a0 ? (b0 - a0) % s : (s - (a0 - b0) % s) % s;  // b's column in a's rows
  return d < a.width || d + b.width > s;
}

inline bool same(const Rows &a, const Rows &b) { return a.p == b.p && a.stride == b.stride; }

}  // namespace rglru
