// Quantization of bf16 rows to 8-bit integers, one fp32 scale a row (the rule:
// int8_rule.h), from dense rows x [T, K] or from the gather itself: with int8
// projection weights the staged rows never reach memory.
//
// Bound: HBM, 2 bytes in and 1 out per element; for few rows a launch and one
// trip to memory (two with a gather: ids, then rows). A row is owned by TPR
// threads, each with P pieces of 8 elements in registers between the maximum
// and the codes: one pass over memory. The maximum is taken on the bit
// patterns (exact, any order).
#include <algorithm>

#include "common.h"
#include "fp8_table.h"
#include "int8_rule.h"

namespace engram {

namespace {

enum Source { kDense, kTable, kTableFp8 };

struct Int8QArgs {
  const void* src;           // x [T, K], or a table of rows
  const uint8_t* scales;     // fp8 table: E8M0 [num_rows, head_dim / 32]
  int64_t num_rows;
  const int32_t* ids;
  int64_t st, sc;
  int head_dim;
  int64_t T;
  int K;
  uint8_t* xq;
  float* xs;
  int32_t* err;
};

__device__ __forceinline__ uint4 piece_of(const Int8QArgs& a, int src, int64_t t, int p, bool& bad) {
  if (src == kDense) return reinterpret_cast<const uint4*>(a.src)[t * (a.K / 8) + p];
  const int ppc = a.head_dim / 8, c = p / ppc, part = p - c * ppc;
  const int64_t id = a.ids[t * a.st + (int64_t)c * a.sc];
  if (id < 0 || id >= a.num_rows) {
    bad = true;
    return make_uint4(0, 0, 0, 0);
  }
  if (src == kTable) return reinterpret_cast<const uint4*>(a.src)[id * ppc + part];
  const uint2 codes = reinterpret_cast<const uint2*>(a.src)[id * ppc + part];
  const float s = e8m0_to_f32(a.scales[(id * ppc + part) / 4]);
  uint32_t o[4];
  fp8_word_to_bf16(codes.x, s, o);
  fp8_word_to_bf16(codes.y, s, o + 2);
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int SRC, int P, int TPR>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void int8_quantize_kernel(const Int8QArgs a) {
  constexpr int BS = TPR < 256 ? 256 : TPR, RPB = BS / TPR, WPR = TPR / 64;
  __shared__ uint32_t red[BS / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t t = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * RPB + wave / WPR;
  const bool live = t < a.T;                       // uniform per wave
  const int pieces = a.K / 8, i0 = tid % TPR;
  bool bad = false;
  uint4 v[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    v[p] = make_uint4(0, 0, 0, 0);
    if (live && i0 + p * TPR < pieces) v[p] = piece_of(a, SRC, t, i0 + p * TPR, bad);
  }
  if (SRC != kDense && bad && a.err) atomicOr(a.err, 1);
  uint32_t m = 0;
#pragma unroll
  for (int p = 0; p < P; ++p) m = int8_amax8(v[p], m);
  m = int8_wave_amax(m);
  if constexpr (WPR > 1) {
    if (lane == 0) red[wave] = m;
    __syncthreads();
    const int w0 = wave / WPR * WPR;
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = max(m, red[w0 + w]);
  }
  if (!live) return;
  const Int8Row r = int8_row(m, 1.f);
#pragma unroll
  for (int p = 0; p < P; ++p) {
    if (i0 + p * TPR >= pieces) break;
    reinterpret_cast<uint2*>(a.xq)[t * pieces + i0 + p * TPR] = int8_codes8(v[p], r);
  }
  if (i0 == 0) a.xs[t] = r.scale;
}

template <int SRC, int P, int TPR>
hipError_t launch(const Int8QArgs& a, hipStream_t s) {
  constexpr int BS = TPR < 256 ? 256 : TPR, RPB = BS / TPR;
  // a grid dimension holds fewer than 2^32 threads
  const int64_t blocks = (a.T + RPB - 1) / RPB, gx = std::min<int64_t>(blocks, 1 << 20);
  hipLaunchKernelGGL((int8_quantize_kernel<SRC, P, TPR>), dim3((uint32_t)gx, (uint32_t)((blocks + gx - 1) / gx)),
                     dim3(BS), 0, s, a);
  return hipGetLastError();
}

// Few rows: one piece a thread where that makes a workgroup, for latency. Many:
// four a thread, more bytes in flight a wave. K < 2^17: 16384 pieces.
template <int SRC>
hipError_t run(const Int8QArgs& a, hipStream_t s) {
  const int pieces = a.K / 8;
  if (pieces <= 64) return launch<SRC, 1, 64>(a, s);
  if (a.T <= dev_info().num_cus) {
    if (pieces <= 256) return launch<SRC, 1, 256>(a, s);
    if (pieces <= 1024) return launch<SRC, 1, 1024>(a, s);
  }
  if (pieces <= 256) return launch<SRC, 4, 64>(a, s);
  if (pieces <= 1024) return launch<SRC, 4, 256>(a, s);
  if (pieces <= 4096) return launch<SRC, 4, 1024>(a, s);
  return launch<SRC, 16, 1024>(a, s);
}

}  // namespace

hipError_t launch_int8_quantize(const void* x, int64_t T, int K, uint8_t* xq, float* xs, hipStream_t s) {
  return run<kDense>({x, nullptr, 0, nullptr, 0, 0, 0, T, K, xq, xs, nullptr}, s);
}

hipError_t launch_gather_int8(const void* table, const uint8_t* table_scales, int64_t num_rows, int head_dim,
                              const int32_t* ids, int64_t st, int64_t sc, int64_t T, int n_cols, uint8_t* xq, float* xs,
                              int32_t* err, hipStream_t s) {
  const Int8QArgs a{table, table_scales, num_rows, ids, st, sc, head_dim, T, n_cols * head_dim, xq, xs, err};
  return table_scales ? run<kTableFp8>(a, s) : run<kTable>(a, s);
}

}  // namespace engram
