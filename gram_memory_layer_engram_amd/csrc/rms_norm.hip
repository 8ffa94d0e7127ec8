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
// 1 + 1/32 of codes and scale; the weight row comes from L2. 8192 tokens of
// four streams of 4096 with a residual: MXFP8 output 131-134 us (742 MB, 5.6
// TB/s; leaving out the quantizer's arithmetic or the scale bytes changes it
// by 1%), bf16 output 177 us (1.07 GB, 6.1 TB/s), both 203 us (1.21 GB, 6.0
// TB/s). One token: 3.0 us, a launch and one trip to memory. Without profit:
// workgroups regrouped so that a token's copies share an XCD's L2 (the same
// time), non-temporal loads of the residual (3% faster on these 268 MB, 17%
// slower where it lies in the Infinity Cache).
//
// Layout: a row is owned by TPR threads. Each of its waves takes a contiguous
// run of P * 64 pieces of 8 elements, lane l the pieces l, 64 + l, .. of the
// run (16-byte loads, contiguous over the wave), all kept in registers between
// the sum and the outputs: one pass over memory. Waves of one row add their
// sums through LDS in wave order. An MX block is 4 neighbouring lanes' pieces:
// its maximum is two quad permutations; the scale bytes of a wave's run (16 a
// piece) are contiguous and leave as one store of 16 * P bytes through LDS.
// Outputs go non-temporal: the kernel never reads them back.
#include <algorithm>

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

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void store16_nt(uint16_t* dst, const uint4& v) {
  const u32x4 w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(dst));
}

// v of the lane whose index differs in bit 0 (bit 1): quad permutations
// [1,0,3,2] and [2,3,0,1].
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true);
}

// Pointers are not __restrict__: residual_out may be residual and out may be
// x; a thread reads all of its pieces before it writes any of them.
template <int P, int TPR>
__global__ __launch_bounds__(TPR < 256 && 256 % TPR == 0 ? 256 : TPR) void add_rms_norm_kernel(const RmsNormArgs a) {
  constexpr int BS = TPR < 256 && 256 % TPR == 0 ? 256 : TPR;
  constexpr int RPB = BS / TPR;                    // rows per workgroup
  constexpr int WPR = TPR / 64;                    // waves per row
  __shared__ float red[BS / 64];
  __shared__ uint8_t sbytes[BS / 64][16 * P];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + wave / WPR;
  const bool live = row < a.rows;                  // uniform per wave
  const int64_t t = live ? row / a.hc : 0;
  const int h = live ? (int)(row - t * a.hc) : 0;
  const int pieces = a.dim / 8;
  const int i0 = wave % WPR * (P * 64) + lane;     // this lane's first piece
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.x_st + h * a.x_sh) + i0;
  const uint4* rr = reinterpret_cast<const uint4*>(a.residual + t * a.r_st + h * a.r_sh) + i0;

  float s[P][8];
  uint4 xv[P], rv[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    xv[p] = rv[p] = make_uint4(0, 0, 0, 0);
    if (live && i0 + p * 64 < pieces) {
      xv[p] = xr[p * 64];
      if (a.residual) rv[p] = rr[p * 64];
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    unpack8(xv[p], s[p]);
    if (a.residual) {
      float r8[8];
      unpack8(rv[p], r8);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[p][e] += r8[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(s[p][e], s[p][e], sum);
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

  const uint4* wr = reinterpret_cast<const uint4*>(a.weight + (int64_t)(a.weight_hc > 1 ? h : 0) * a.dim) + i0;
  const int64_t base = row * pieces + i0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    // the four lanes of an MX block are live together (dim % 32 == 0 then)
    if (i0 + p * 64 >= pieces) break;
    if (a.residual_out) store16_nt(a.residual_out + (base + p * 64) * 8, pack8(s[p]));
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = s[p][e] * inv;
    if (a.weight) {
      float w8[8];
      unpack8(wr[p * 64], w8);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] *= w8[e];
    }
    if (a.out) store16_nt(a.out + (base + p * 64) * 8, pack8(y));
    if (a.xq) {
      uint32_t amax = 0;   // magnitudes order like unsigned integers, NaN above infinity
#pragma unroll
      for (int e = 0; e < 8; ++e) amax = max(amax, __float_as_uint(y[e]) & 0x7fffffffu);
      amax = max(amax, quad_xor1(amax));
      amax = max(amax, quad_xor2(amax));
      uint32_t packed[2];
      const int byte = mx_piece_f32(y, amax, packed);
      const u32x2 c = {packed[0], packed[1]};
      __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(a.xq + (base + p * 64) * 8));
      if ((lane & 3) == 0) sbytes[wave][p * 16 + (lane >> 2)] = (uint8_t)byte;
    }
  }
  if (a.xq) {
    // the run's scale bytes: written and read by this wave alone
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int n = min(P * 64, pieces - wave % WPR * (P * 64)) / 4;   // bytes of the run (negative: none)
    uint8_t* dst = a.xs + (row * pieces + wave % WPR * (P * 64)) / 4;
    if (lane < n) {
#pragma unroll
      for (int k = 0; k < (P + 3) / 4; ++k)
        if (lane + 64 * k < n) dst[lane + 64 * k] = sbytes[wave][lane + 64 * k];
    }
  }
}

template <int P, int TPR>
hipError_t launch(const RmsNormArgs& a, hipStream_t s) {
  constexpr int BS = TPR < 256 && 256 % TPR == 0 ? 256 : TPR, RPB = BS / TPR;
  // a grid dimension holds fewer than 2^32 threads: past 2^20 workgroups the
  // rows run on into y
  const int64_t blocks = (a.rows + RPB - 1) / RPB, gx = std::min<int64_t>(blocks, 1 << 20);
  hipLaunchKernelGGL((add_rms_norm_kernel<P, TPR>), dim3((uint32_t)gx, (uint32_t)((blocks + gx - 1) / gx)), dim3(BS),
                     0, s, a);
  return hipGetLastError();
}

}  // namespace

// Few rows: latency counts, one piece a thread (T 1, four rows of 4096: 3.1 us
// with 512 threads a row, 3.7 with 256). Many: four pieces a thread keep more
// bytes in flight per wave.
hipError_t launch_add_rms_norm(const RmsNormArgs& a, hipStream_t s) {
  const int pieces = a.dim / 8;
  if (pieces <= 64) return launch<1, 64>(a, s);
  if (a.rows <= dev_info().num_cus) {
    if (pieces <= 128) return launch<1, 128>(a, s);
    if (pieces <= 256) return launch<1, 256>(a, s);
    if (pieces <= 512) return launch<1, 512>(a, s);
    if (pieces <= 1024) return launch<1, 1024>(a, s);
    return launch<2, 1024>(a, s);   // dim <= 16384
  }
  if (pieces <= 128) return launch<2, 64>(a, s);
  if (pieces <= 256) return launch<4, 64>(a, s);
  if (pieces <= 512) return launch<4, 128>(a, s);
  if (pieces <= 1024) return launch<4, 256>(a, s);
  return launch<4, 512>(a, s);
}

}  // namespace engram
