// rglru_e4m3.h -- cached rows as e4m3 values with a power-of-two scale for each (token, head).
//
// A row x of dh values is stored as c_i = e4m3(x_i / s) and s, s the smallest power of two with max |x| / s <= 448
// (e4m3's largest value), 2^-117 at least, as e8m0 (its exponent + 127 in a byte). Division by a power of two is
// exact, so there is one rounding, of x_i / s to the nearest e4m3 value (ties to even), and the result is defined to
// the bit; a finer scale would not make it smaller, as e4m3's steps are relative. Every c_i s is a multiple of 2^-126:
// a normal number, exact in bf16 and in fp32. A row with an infinity or a NaN gets the scale 255, which is NaN.
#pragma once

#include "rglru_mfma.h"

namespace rglru {

constexpr int kScaleMin = 127 - 117;  // the least stored exponent
constexpr int kScaleNan = 255;

// The stored exponent for a row whose largest magnitude has these fp32 bits (a NaN's are above infinity's).
__device__ __forceinline__ unsigned scale_of(unsigned top) {
  if (top >= 0x7F800000u) return kScaleNan;
  // 448 = 1.75 * 2^8: one more where the significand is above 1.75
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<unsigned>(max(e, kScaleMin));
}

// 1 / s, for the exponents that scale_of gives (7 .. 244 as exponents of fp32)
__device__ __forceinline__ float inverse_scale(unsigned b) { return __uint_as_float((254u - b) << 23); }

// What a stored exponent stands for, any byte: 0 is 2^-127, 255 NaN.
__device__ __forceinline__ float scale_value(unsigned b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == kScaleNan ? 0x7FC00000u : b << 23);
}

// Four values as e4m3, the first in the lowest byte.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
  int w = 0;
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return static_cast<uint32_t>(w);
}

typedef __bf16 bf16x2_v __attribute__((ext_vector_type(2)));

// Two neighbouring codes of a word (its low or high half) times s, as bf16: exact (see above). The instruction
// takes the scale as an fp32 whose exponent alone counts.
template <bool HIGH> __device__ __forceinline__ uint32_t bf16x2_of(uint32_t codes, float s) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, s, HIGH));
}

}  // namespace rglru
