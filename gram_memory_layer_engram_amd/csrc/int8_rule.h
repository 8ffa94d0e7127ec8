// Rows in 8-bit integers with one fp32 scale a row, used by the quantizers
// (int8q.hip) and by the norm's 8-bit output (post_pre_norm.hip).
//
// For a row v with largest magnitude a:
//   scale = a / 127              (fp32, rounded once)
//   code  = rne(v * (127 / a))   (fp32 quotient and product, each rounded once)
// so codes lie in -127..127 and code * scale is within half a step of v, plus
// the two fp32 roundings. a = 0: scale 0, codes 0. A row with an infinity or a
// NaN has no finite maximum: scale NaN and codes 0, so that every product of
// the row is NaN. Where a < 2^-100 the row is first multiplied by 2^100
// (exact), for 127 / a would overflow; its scale may be subnormal.
#pragma once

#include "common.h"

namespace engram {

struct Int8Row {
  float pre, inv;   // code = rne((v * pre) * inv)
  float scale;
};

// From the bits of the largest magnitude (magnitudes order like unsigned
// integers, NaN above infinity). scale = (a * factor) / 127: a norm takes its
// row's codes from values that its factor 1 / rms is left out of.
__device__ __forceinline__ Int8Row int8_row(uint32_t amax, float factor) {
#pragma clang fp contract(off)
  if (amax >= 0x7f800000u) return {0.f, 0.f, __uint_as_float(0x7fc00000u)};
  const float a = __uint_as_float(amax);
  const float pre = a < 0x1p-100f ? 0x1p100f : 1.f;
  return {pre, amax ? 127.f / (a * pre) : 0.f, a * factor / 127.f};
}

// Four codes, v[0] in the low byte. Adding 1.5 * 2^23 rounds to a whole number,
// nearest-even, and leaves its two's complement in the low byte.
__device__ __forceinline__ uint32_t int8_codes4(const float* v, const Int8Row& r) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a row without a finite maximum: 0 * NaN would leave a NaN's bits
    const float q = r.inv == 0.f ? 0.f : (v[i] * r.pre) * r.inv;
    b[i] = __float_as_uint(q + 12582912.f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return lo | hi;
}

}  // namespace engram
