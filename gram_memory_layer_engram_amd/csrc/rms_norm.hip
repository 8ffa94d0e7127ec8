// Residual addition and root-mean-square norm of the layer's streams, with
// the norm's output in bf16, in MXFP8, or both.
//
// "vllm.models.deepseek_v4_1.common.engram", Engram.__init__ / forward: the
// layer updates hidden [T, hc_mult, dim] and carries rms_norm_eps; what
// follows it adds a branch to the streams and normalizes them. Per row (t, h):
//   s   = x + residual                     (fp32; residual_out = bf16(s))
//   inv = 1 / sqrt(sum(s^2) / dim + eps)
//   y   = s * inv * weight[h]
//   out = bf16(y), and / or per 32 consecutive elements the OCP MX v1.0
//   conversion of y to MXFP8-E4M3 (the rule of mxq.hip, on fp32 values).
// Everything up to the outputs stays in fp32: the norm is taken of the
// unrounded sum and the codes are rounded once from y, so neither the stored
// stream's rounding nor a bf16 y's is in them.
//
// Bound: HBM. Per element 2 bytes of x, 4 of residual in and out, 2 of out or
// 1 + 1/32 of codes and scale; the weight row comes from L2.
//
// Layout: TPR threads own a row, each P pieces of 8 elements at a stride of
// TPR pieces (16-byte loads, contiguous over a wave), all kept in registers
// between the sum and the outputs: one pass over memory. A wave owns a row up
// to dim 64*8*P; longer rows add their waves' sums through LDS in wave order.
// An MX block is 4 neighbouring lanes' pieces: its maximum is two exchanges.
#include "common.h"
#include "mx_rule.h"

namespace engram {

namespace {

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  f[0] = bf16lo(v.x); f[1] = bf16hi(v.x);
  f[2] = bf16lo(v.y); f[3] = bf16hi(v.y);
  f[4] = bf16lo(v.z); f[5] = bf16hi(v.z);
  f[6] = bf16lo(v.w); f[7] = bf16hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(cvt_pk_bf16(f[0], f[1]), cvt_pk_bf16(f[2], f[3]), cvt_pk_bf16(f[4], f[5]),
                    cvt_pk_bf16(f[6], f[7]));
}

// Pointers are not __restrict__: residual_out may be residual and out may be
// x; a thread reads all of its pieces before it writes any of them.
template <int P, int TPR>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void add_rms_norm_kernel(const RmsNormArgs a) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;   // rows per workgroup
  constexpr int WPR = TPR / 64;                    // waves per row
  __shared__ float red[RPB * WPR];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int in_row = tid % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + tid / TPR;
  const bool live = row < a.rows;
  const int64_t t = live ? row / a.hc : 0;
  const int h = live ? (int)(row - t * a.hc) : 0;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.x_st + h * a.x_sh);
  const uint4* rr = a.residual ? reinterpret_cast<const uint4*>(a.residual + t * a.r_st + h * a.r_sh) : nullptr;
  const uint4* wr = a.weight ? reinterpret_cast<const uint4*>(a.weight + (int64_t)(a.weight_hc > 1 ? h : 0) * a.dim)
                             : nullptr;
  const int pieces = a.dim / 8;

  float s[P][8];
  uint4 xv[P], rv[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    xv[p] = rv[p] = make_uint4(0, 0, 0, 0);
    const int i = p * TPR + in_row;
    if (live && i < pieces) {
      xv[p] = xr[i];
      if (rr) rv[p] = rr[i];
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float r8[8];
    unpack8(xv[p], s[p]);
    unpack8(rv[p], r8);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (rr) s[p][e] += r8[e];
      sum = fmaf(s[p][e], s[p][e], sum);
    }
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
  if constexpr (WPR > 1) {
    if (lane == 0) red[wave] = sum;
    __syncthreads();
    const int w0 = wave / WPR * WPR;
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) sum += red[w0 + w];
  }
  const float inv = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
  if (!live) return;

  const int64_t base = row * pieces;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int i = p * TPR + in_row;
    // the four lanes of an MX block are live together (dim % 32 == 0 then)
    if (i >= pieces) break;
    if (a.residual_out) reinterpret_cast<uint4*>(a.residual_out)[base + i] = pack8(s[p]);
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = s[p][e] * inv;
    if (wr) {
      float w8[8];
      unpack8(wr[i], w8);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= w8[e];
    }
    if (a.out) reinterpret_cast<uint4*>(a.out)[base + i] = pack8(y);
    if (a.xq) {
      uint32_t amax = 0;   // magnitudes order like unsigned integers, NaN above infinity
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 1, 64));
      amax = max(amax, (uint32_t)__shfl_xor((int)amax, 2, 64));
      uint32_t packed[2];
      const int byte = mx_piece_f32(y, amax, packed);
      reinterpret_cast<uint2*>(a.xq)[base + i] = make_uint2(packed[0], packed[1]);
      if ((lane & 3) == 0) a.xs[(base + i) >> 2] = (uint8_t)byte;
    }
  }
}

template <int P, int TPR>
hipError_t launch(const RmsNormArgs& a, hipStream_t s) {
  constexpr int RPB = TPR < 256 ? 256 / TPR : 1;
  constexpr int BS = TPR < 256 ? 256 : TPR;
  hipLaunchKernelGGL((add_rms_norm_kernel<P, TPR>), dim3((uint32_t)((a.rows + RPB - 1) / RPB)), dim3(BS), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_add_rms_norm(const RmsNormArgs& a, hipStream_t s) {
  const int pieces = a.dim / 8;
  if (pieces <= 64) return launch<1, 64>(a, s);
  if (pieces <= 128) return launch<2, 64>(a, s);
  if (pieces <= 256) return launch<1, 256>(a, s);
  if (pieces <= 512) return launch<2, 256>(a, s);
  if (pieces <= 1024) return launch<4, 256>(a, s);
  return launch<8, 256>(a, s);   // dim <= 16384
}

}  // namespace engram
