// MXFP4 weights expanded to bf16 and MXFP8 activations back to bf16, for the
// bf16 GEMM, where the GEMMs on the codes do not apply (K % 256 == 128 past
// the GEMV's token counts).
//
// Format (OCP Microscaling Formats v1.0): e2m1 codes, two per byte with the
// lower k in the low nibble, W[N, K/2], and one E8M0 byte per row and 32 k,
// S[N, K/32]; the value of a code is e2m1(c) * 2^(byte - 127) (byte 255: NaN).
// e2m1 has 2 significant bits and e4m3 has 4, so both products are exact in
// bf16 (its 8 bits and fp32's exponent range; past the top they become inf).
//
// Bound: HBM / L2 writes of the expanded weight, 2 bytes of each 2.53 moved (N
// 20480, K 2048, 84 MB written: about 20 us in front of a GEMM of 490); a
// thread turns one 4-byte word of codes (8 weights) into one 16-byte piece, so
// stores are contiguous over a wave.
#include <algorithm>

#include "common.h"
#include "fp8_table.h"

namespace engram {

namespace {

// Word i of a row-major code matrix covers k 8*i .. 8*i+7 of its row: scale
// byte i / 4 of the flattened scales.
__global__ __launch_bounds__(256) void mxfp4_to_bf16_kernel(const uint32_t* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t words,
                                                            uint4* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < words; i += (int64_t)gridDim.x * 256) {
    const uint32_t c = codes[i];
    const float s = __uint_as_float((uint32_t)scales[i >> 2] << 23);   // the conversion reads the exponent field
    uint4 o;
    o.x = fp4_pair_to_bf16<0>(c, s);
    o.y = fp4_pair_to_bf16<1>(c, s);
    o.z = fp4_pair_to_bf16<2>(c, s);
    o.w = fp4_pair_to_bf16<3>(c, s);
    out[i] = o;
  }
}

// 8 codes of an MXFP8 row -> 8 bf16.
__global__ __launch_bounds__(256) void mxfp8_to_bf16_kernel(const uint2* __restrict__ codes,
                                                            const uint8_t* __restrict__ scales, int64_t pieces,
                                                            uint4* __restrict__ out) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < pieces; i += (int64_t)gridDim.x * 256) {
    const uint2 c = codes[i];
    const float s = e8m0_to_f32(scales[i >> 2]);
    uint32_t o[4];
    fp8_word_to_bf16(c.x, s, o);
    fp8_word_to_bf16(c.y, s, o + 2);
    out[i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

uint32_t blocks_for(int64_t n) { return (uint32_t)std::min<int64_t>((n + 255) / 256, 1 << 20); }

}  // namespace

hipError_t launch_mxfp4_to_bf16(const void* w, const uint8_t* scales, int64_t N, int K, void* out, hipStream_t s) {
  const int64_t words = N * (K / 8);
  hipLaunchKernelGGL(mxfp4_to_bf16_kernel, dim3(blocks_for(words)), dim3(256), 0, s,
                     (const uint32_t*)w, scales, words, (uint4*)out);
  return hipGetLastError();
}

hipError_t launch_mxfp8_to_bf16(const uint8_t* xq, const uint8_t* xs, int64_t T, int K, void* out, hipStream_t s) {
  const int64_t pieces = T * (K / 8);
  hipLaunchKernelGGL(mxfp8_to_bf16_kernel, dim3(blocks_for(pieces)), dim3(256), 0, s,
                     (const uint2*)xq, xs, pieces, (uint4*)out);
  return hipGetLastError();
}

}  // namespace engram
