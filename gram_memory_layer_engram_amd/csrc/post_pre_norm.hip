// The norm after a block, its gate, the scaled residual and the norm before the
// next block, in one pass over the streams.
//
// The layer's streams are [T, hc, dim], its branch is gated per token and copy. A
// block between two norms adds to a stream, per row (t, h):
//   p   = x / sqrt(sum(x^2) / dim + post_eps) * post_weight[h]
//   s   = residual_scale * residual + branch_scale * (g * p)
//   y   = s / sqrt(sum(s^2) / dim + eps) * pre_weight[h]
// residual_out = bf16(s); y leaves in bf16, in MXFP8 (the rule of mx_rule.h) or
// as int8 codes with one scale a row (int8_rule.h), bf16 beside either. g is one
// factor a row or one a channel, as it is or through a sigmoid. Everything up to
// the outputs stays in fp32, each output is rounded once from there, and sums run
// in a fixed order.
//
// The int8 codes come from s * pre_weight and that row's maximum, taken in the
// same reduction as sum(s^2): 1 / rms cancels in them and is in the scale alone.
//
// Layout: as rms_norm.hip. A row is owned by TPR threads, each wave a contiguous
// run of P * 64 pieces of 8 elements, all of x, residual, gate and both weights
// in registers before the first sum: one pass, two reductions.
//
// Bound: HBM. Per element 2 bytes of x, 4 of the stream in and out, 2 of a channel
// gate, 2 of out or 1 and a bit of codes; weights come from L2. 8192 tokens of four
// streams of 4096, x of its own for each: int8 162 us (939 MB, 5.8 TB/s), bf16 181 us
// (5.9); one x for four streams, MXFP8 142-147 us (742 MB, 5.1), bf16 157 (5.6): there
// the rows' own latency shows, 16 waves a compute unit with both sums to wait for. One
// token: 3.8 us, a launch, one trip to memory and two sums.
// Without profit: the weights loaded behind the first sum (fewer registers: 2-8%
// slower); one workgroup for the copies that share x, its norm taken once, the next
// copy's operands in flight (163 us); a persistent grid with the next row in flight and
// the weights kept in registers (161 us); larger and smaller workgroups.
#include <algorithm>

#include "common.h"
#include "int8_rule.h"
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

// v of the lane whose index differs in bit 0 (bit 1): quad permutations.
__device__ __forceinline__ uint32_t quad_xor1(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t quad_xor2(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true);
}

// exp as a power of two on the hardware's v_exp_f32, reciprocal on v_rcp_f32 (1 ulp
// each). z * log2(e) is rounded in units of its own size: the sigmoid is within 2^-20
// of its value for |z| < 11, 2^-19 to 16 and 2^-17 to 80 (measured 0.63, 1.05 and 4.0 of
// 2^-20), far under a bf16 step. With expf, within 2^-21 everywhere, the norms with a
// channel gate take longer: one token of 4096 3.9 -> 4.2 us, 1037 of 7168 19.5 -> 20.6,
// 4096 of 4096 31.1 -> 32.1.
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, off, 64));
  return v;
}

// A barrier for LDS alone: __syncthreads() also waits for every store in flight.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Pointers are not __restrict__: residual_out may be residual and out may be
// x; a thread reads all of its pieces before it writes any of them.
template <int P, int TPR>
__global__ __launch_bounds__(TPR < 256 && 256 % TPR == 0 ? 256 : TPR) void post_pre_norm_kernel(const PostPreNormArgs a) {
  constexpr int BS = TPR < 256 && 256 % TPR == 0 ? 256 : TPR;
  constexpr int RPB = BS / TPR;                    // rows per workgroup
  constexpr int WPR = TPR / 64;                    // waves per row
  __shared__ float red[2][BS / 64];
  __shared__ uint32_t redm[BS / 64];
  __shared__ uint8_t sbytes[BS / 64][16 * P];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int w0 = wave / WPR * WPR;                 // the row's first wave
  const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + wave / WPR;
  const bool live = row < a.rows;                  // uniform per wave
  const int64_t t = live ? row / a.hc : 0;
  const int h = live ? (int)(row - t * a.hc) : 0;
  const int pieces = a.dim / 8;
  const int i0 = wave % WPR * (P * 64) + lane;     // this lane's first piece
  const bool channel = a.gate_format == kGateChannel;
  const uint4* xr = reinterpret_cast<const uint4*>(a.x + t * a.x_st + h * a.x_sh) + i0;
  const uint4* rr = reinterpret_cast<const uint4*>(a.residual + t * a.r_st + h * a.r_sh) + i0;
  const uint4* gr = reinterpret_cast<const uint4*>((const uint16_t*)a.gate + t * a.g_st + h * a.g_sh) + i0;
  const uint4* w1 = reinterpret_cast<const uint4*>(a.post_weight + (int64_t)(a.post_hc > 1 ? h : 0) * a.dim) + i0;
  const uint4* w2 = reinterpret_cast<const uint4*>(a.pre_weight + (int64_t)(a.pre_hc > 1 ? h : 0) * a.dim) + i0;

  uint4 xv[P], rv[P], gv[P], pv[P], qv[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    xv[p] = rv[p] = gv[p] = pv[p] = qv[p] = make_uint4(0, 0, 0, 0);
    if (live && i0 + p * 64 < pieces) {
      xv[p] = xr[p * 64];
      if (a.residual) rv[p] = rr[p * 64];
      if (channel) gv[p] = gr[p * 64];
      if (a.post_weight) pv[p] = w1[p * 64];
      if (a.pre_weight) qv[p] = w2[p * 64];
    }
  }
  float rg = a.branch_scale;   // every factor of the row
  if (a.gate_format == kGateRow && live) {
    const float g = ((const float*)a.gate)[t * a.g_st + h * a.g_sh];
    rg *= a.sigmoid ? sigmoid(g) : g;
  }

  float s[P][8];
  float sum = 0.f;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    unpack8(xv[p], s[p]);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(s[p][e], s[p][e], sum);
  }
  if (a.post_norm) {
    sum = wave_sum(sum);
    if constexpr (WPR > 1) {
      if (lane == 0) red[0][wave] = sum;
      lds_barrier();
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < WPR; ++w) sum += red[0][w0 + w];
    }
    rg *= 1.0f / sqrtf(sum / (float)a.dim + a.post_eps);
  }

  // s, stored at once, and in its place s * pre_weight
  sum = 0.f;
  const int64_t base = row * pieces + i0;
  uint32_t amax[P];   // magnitudes order like unsigned integers, NaN above infinity
#pragma unroll
  for (int p = 0; p < P; ++p) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) s[p][e] *= rg;
    if (a.post_weight) {
      unpack8(pv[p], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[p][e] *= f[e];
    }
    if (channel) {
      unpack8(gv[p], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[p][e] *= a.sigmoid ? sigmoid(f[e]) : f[e];
    }
    if (a.residual) {
      unpack8(rv[p], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[p][e] = fmaf(a.residual_scale, f[e], s[p][e]);
    }
    if (a.residual_out && live && i0 + p * 64 < pieces) store16_nt(a.residual_out + (base + p * 64) * 8, pack8(s[p]));
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(s[p][e], s[p][e], sum);
    if (a.pre_weight) {
      unpack8(qv[p], f);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[p][e] *= f[e];
    }
    amax[p] = 0;
    if (a.q_format == kQInt8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) amax[p] = max(amax[p], __float_as_uint(s[p][e]) & 0x7fffffffu);
    }
  }
  sum = wave_sum(sum);
  uint32_t rmax = 0;
  if (a.q_format == kQInt8) {
#pragma unroll
    for (int p = 0; p < P; ++p) rmax = max(rmax, amax[p]);
    rmax = wave_max(rmax);
  }
  if constexpr (WPR > 1) {
    if (lane == 0) {
      red[1][wave] = sum;
      redm[wave] = rmax;
    }
    lds_barrier();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      sum += red[1][w0 + w];
      rmax = max(rmax, redm[w0 + w]);
    }
  }
  const float inv2 = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
  if (!live) return;

  const Int8Row q8 = int8_row(rmax, inv2);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    // the four lanes of an MX block are live together (dim % 32 == 0 then)
    if (i0 + p * 64 >= pieces) break;
    if (a.q_format == kQInt8) {
      const uint2 q = int8_codes8(s[p], q8);
      const u32x2 c = {q.x, q.y};
      __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(a.xq + (base + p * 64) * 8));
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[p][e] *= inv2;
    if (a.out) store16_nt(a.out + (base + p * 64) * 8, pack8(s[p]));
    if (a.q_format == kQMx) {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(s[p][e]) & 0x7fffffffu);
      m = max(m, quad_xor1(m));
      m = max(m, quad_xor2(m));
      uint32_t packed[2];
      const int byte = mx_piece_f32(s[p], m, packed);
      const u32x2 c = {packed[0], packed[1]};
      __builtin_nontemporal_store(c, reinterpret_cast<u32x2*>(a.xq + (base + p * 64) * 8));
      if ((lane & 3) == 0) sbytes[wave][p * 16 + (lane >> 2)] = (uint8_t)byte;
    }
  }
  if (a.q_format == kQInt8) {
    if (i0 == 0) ((float*)a.xs)[row] = q8.scale;
  } else if (a.q_format == kQMx) {
    // the run's scale bytes: written and read by this wave alone
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int n = min(P * 64, pieces - wave % WPR * (P * 64)) / 4;   // bytes of the run (negative: none)
    uint8_t* dst = (uint8_t*)a.xs + (row * pieces + wave % WPR * (P * 64)) / 4;
#pragma unroll
    for (int k = 0; k < (P + 3) / 4; ++k)
      if (lane + 64 * k < n) dst[lane + 64 * k] = sbytes[wave][lane + 64 * k];
  }
}

template <int P, int TPR>
hipError_t launch(const PostPreNormArgs& a, hipStream_t s) {
  constexpr int BS = TPR < 256 && 256 % TPR == 0 ? 256 : TPR, RPB = BS / TPR;
  // a grid dimension holds fewer than 2^32 threads: past 2^20 workgroups the
  // rows run on into y
  const int64_t blocks = (a.rows + RPB - 1) / RPB, gx = std::min<int64_t>(blocks, 1 << 20);
  hipLaunchKernelGGL((post_pre_norm_kernel<P, TPR>), dim3((uint32_t)gx, (uint32_t)((blocks + gx - 1) / gx)), dim3(BS),
                     0, s, a);
  return hipGetLastError();
}

}  // namespace

// Few rows: latency counts, one piece a thread (T 61, four rows of 2048 bf16: 3.7 us,
// two pieces 4.1). Some more: two (400 rows of 4096: 4.9, four pieces 5.8, one 5.5).
// Many: four keep more bytes in flight per wave (2000 rows of 4096 mxfp8 10.5, two
// 11.5).
hipError_t launch_post_pre_norm(const PostPreNormArgs& a, hipStream_t s) {
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
  if (a.rows <= 3 * dev_info().num_cus) {
    if (pieces <= 256) return launch<2, 128>(a, s);
    if (pieces <= 512) return launch<2, 256>(a, s);
    if (pieces <= 1024) return launch<2, 512>(a, s);
    return launch<2, 1024>(a, s);
  }
  if (pieces <= 256) return launch<4, 64>(a, s);
  if (pieces <= 512) return launch<4, 128>(a, s);
  if (pieces <= 1024) return launch<4, 256>(a, s);
  return launch<4, 512>(a, s);
}

}  // namespace engram
