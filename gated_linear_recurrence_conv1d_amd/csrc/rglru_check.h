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

// ---- operators on rows of heads
constexpr long long kMaxStride = 1LL << 20;  // elements from token to token
constexpr long long kMaxTokens = 0x7FFFFF00;  // token and cache row indices stay in an int

inline Rows heads_of(const void *p, size_t rows, int heads, int dh, long long stride, rglru_dtype dt) {
  const size_t e = elem_bytes(dt);
  return {p, rows, static_cast<size_t>(heads) * dh * e, static_cast<size_t>(stride) * e};
}

inline Rows flat(const void *p, size_t bytes) { return {p, p ? size_t{1} : 0, bytes, bytes}; }

// Sizes and types every operator on rows of heads shares.
inline rglru_status check_heads(long long rows, int Hq, int Hkv, int dh, rglru_dtype dt) {
  if (rows < 1 || Hq < 1 || Hkv < 1 || dh < 1) return RGLRU_ERR_INVALID_ARG;
  if (dt != RGLRU_F32 && dt != RGLRU_BF16) return RGLRU_ERR_UNSUPPORTED;
  if (Hq > 65535 || Hkv > 65535) return RGLRU_ERR_UNSUPPORTED;
  return RGLRU_OK;
}

inline bool stride_ok(long long stride, int heads, int dh) {
  return stride >= static_cast<long long>(heads) * dh;
}

// The kernels' running maximum starts here: below every score that matters, and finite in exp2
// units.
inline float max_floor(float c) { return -2.9e38f / (c > 1.0f ? c : 1.0f); }

}  // namespace rglru
