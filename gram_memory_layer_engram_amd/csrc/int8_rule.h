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
// nearest-even, and leaves its two's complement in the low byte. ORDINARY: the row
// is finite and needs no factor, its codes are rne(v * inv).
template <bool ORDINARY>
__device__ __forceinline__ uint32_t int8_codes4(const float* v, const Int8Row& r) {
#pragma clang fp contract(off)
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a row without a finite maximum: 0 * NaN would leave a NaN's bits
    const float q = ORDINARY ? v[i] * r.inv : r.inv == 0.f ? 0.f : (v[i] * r.pre) * r.inv;
    b[i] = __float_as_uint(q + 12582912.f);
  }
  const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000c0cu);
  return lo | hi;
}

// Eight codes of fp32 values; of a wave's rows most are ordinary (uniform branch).
__device__ __forceinline__ uint2 int8_codes8(const float* f, const Int8Row& r) {
  if (__all(r.pre == 1.f && r.inv != 0.f)) return make_uint2(int8_codes4<true>(f, r), int8_codes4<true>(f + 4, r));
  return make_uint2(int8_codes4<false>(f, r), int8_codes4<false>(f + 4, r));
}
__device__ __forceinline__ uint2 int8_codes8(const uint4& v, const Int8Row& r) {
  const float f[8] = {bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y), bf16lo(v.z), bf16hi(v.z), bf16lo(v.w), bf16hi(v.w)};
  return int8_codes8(f, r);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Running maximum of the magnitudes of bf16 pairs, each half by itself (bf16
// magnitudes order like unsigned integers).
__device__ __forceinline__ uint32_t int8_amax8(const uint4& v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                               __builtin_bit_cast(u16x2, w[i] & 0x7fff7fffu)));
  return m;
}
// ... and of a wave's, as the bits of an fp32.
__device__ __forceinline__ uint32_t int8_wave_amax(uint32_t m) {
  m = max(m & 0xffffu, m >> 16);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  return m << 16;
}

}  // namespace engram
