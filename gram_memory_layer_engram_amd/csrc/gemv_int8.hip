// Projection in 8-bit integers for small batches, or few rows: kv[T, N] =
// bf16(float(x . W^T) * xs[t] * ws[n]), x int8 with one fp32 scale a token, or (up
// to 16 tokens) bf16, quantized by the rule of int8_rule.h on the way.
//
// With few tokens the product is a stream of the weight, a byte a weight. A
// workgroup owns RT tiles of 16 rows and all T tokens (past 64 a group of 64 or 128
// of them). The sums are whole numbers, exact in any order: k may be split and
// started anywhere, and kv is that of the tiled GEMM bit for bit.
//
// W goes through LDS (gemv_int8_dma.h): a fragment read straight from memory
// touches 16 lines for 64 bytes of each, and the vector cache answers a line per
// clock and lane quarter; a DMA of 8 rows x 128 bytes takes 8 lines whole.
// v_mfma_i32_16x16x64_i8 takes in lane l (row l%16, g = l/16) 16 bytes of k;
// sub-step h of a step is pieces 4h + g of both operands.
//
// Measured (N 20480, K 2048, 42 MB of weight of three in turn; graph replay, 1.8 us
// of it an empty kernel's; a plain read of the same bytes 7.9 us): T 1 / 16 / 32 /
// 48 / 61 in 7.7 / 8.0 / 8.5 / 9.1 / 9.8 us (128x128 GEMM tiles 11.2 - 12.2), from
// bf16 x T 1 / 4 / 8 7.8 / 7.9 / 8.1. Up to 32 tokens that stream bounds it. Beyond,
// x is read by every workgroup from L2 as well, 125 KB each at T 61. Past 64 tokens
// it still beats the GEMM's few tiles: N 12288, K 4096, T 96 / 128 12.0 / 14.1 against
// 20 us, N 4096, K 2048 5.8 / 6.3 against 9.2 - 9.7.
#include <algorithm>

#include "common.h"
#include "gemv_int8_dma.h"
#include "int8_rule.h"

namespace engram {

namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef __attribute__((address_space(3))) void* lds_ptr_t;

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, 0x00020000);
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lgkm0() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" ::: "memory"); }

// Four rows' sums of a token to kv: float(sum) * xs * ws, each step one rounding.
__device__ __forceinline__ void store4(uint16_t* kv, const i32x4& sum, float xs, const f32x4& ws) {
  uint2 o;
  o.x = cvt_pk_bf16((float)sum[0] * xs * ws[0], (float)sum[1] * xs * ws[1]);
  o.y = cvt_pk_bf16((float)sum[2] * xs * ws[2], (float)sum[3] * xs * ws[3]);
  *reinterpret_cast<uint2*>(kv) = o;
}

struct GemvI8Args {
  const void* x;       // int8 [T, K], or bf16 [T, K] (xs null)
  const float* xs;
  const uint8_t* w;
  const float* ws;
  uint16_t* kv;
  int T, K, N;
};

// ---- few tokens (at most 16): x in registers, every wave its own k ----
//
// A wave takes every WAVES-th step, with its x loaded first and the DMAs of DW of
// its STEPS steps of W behind that, in its own ring; no barrier in the loop.
//
// XBF: bf16 x. Every workgroup makes the codes for itself, a wave a token: the
// row, its maximum, its codes into LDS (rows of K bytes, their pieces swapped as
// W's are), while W flies. Twice T * K bytes from L2 for each workgroup, instead
// of a launch.
template <int RT, int WAVES, int DW, int STEPS, bool XBF>
__global__ __launch_bounds__(WAVES * 64) void gemv_int8_reg_kernel(const GemvI8Args a) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int RING = DW * RT * i8::kTileBytes;
  constexpr int KMAX = WAVES * STEPS * i8::kStep, XP = KMAX / 512;   // pieces of 8 a lane holds of a row
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * RT, rows = min(16 * RT, a.N - n0);
  const int g = lane >> 4, r = lane & 15;
  const int t = min(r, a.T - 1);                   // a padding token repeats the last
  const uint32_t K = (uint32_t)a.K;
  const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)rows * K);
  char* xl = lds + WAVES * RING;                   // XBF: codes of T rows, KMAX bytes each, then the scales

  i32x4 xf[STEPS][2];
  uint4 xv[XBF ? XP : 1];
  auto load_row = [&](int tok) {
#pragma unroll
    for (int p = 0; p < XP; ++p) {
      xv[p] = make_uint4(0, 0, 0, 0);
      if (tok < a.T && (p * 64 + lane) * 8 < a.K)
        xv[p] = reinterpret_cast<const uint4*>((const uint16_t*)a.x + (int64_t)tok * a.K)[p * 64 + lane];
    }
  };
  if constexpr (XBF) {
    load_row(wave);
  } else {
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int k = (wave + i * WAVES) * i8::kStep + 64 * h + 16 * g;
        xf[i][h] = i32x4{0, 0, 0, 0};
        if (k < a.K) xf[i][h] = *reinterpret_cast<const i32x4*>((const uint8_t*)a.x + (int64_t)t * a.K + k);
      }
  }
  // what the thread that adds row tile `wave` needs
  const int n = n0 + wave * 16 + 4 * g;
  f32x4 wsc = {0.f, 0.f, 0.f, 0.f};
  if (wave < RT && n < a.N) wsc = *reinterpret_cast<const f32x4*>(a.ws + n);
  float xsc = 0.f;
  if constexpr (!XBF) xsc = a.xs[t];
  __builtin_amdgcn_sched_barrier(0);

  auto issue = [&](int i) {   // a step past the end brings zeros
    const int s = wave + i * WAVES;
    const int slot = wave * RING + i % DW * (RT * i8::kTileBytes);
    const uint32_t kofs = s * i8::kStep < a.K ? (uint32_t)s * i8::kStep : i8::kOob;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int q = 0; q < 2; ++q)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(lds + slot + rt * i8::kTileBytes + q * 1024), 16,
                                                 i8::voffset(lane, rt * 2 + q, kofs, K), 0, 0, 0);
  };
#pragma unroll
  for (int i = 0; i < DW; ++i) issue(i);
  __builtin_amdgcn_sched_barrier(0);

  if constexpr (XBF) {
    float* scales = reinterpret_cast<float*>(xl + a.T * KMAX);
    for (int tok = wave; tok < a.T; tok += WAVES) {
      if (tok >= WAVES) load_row(tok);
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < XP; ++p) m = int8_amax8(xv[p], m);
      const Int8Row q = int8_row(int8_wave_amax(m), 1.f);
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        const int piece = (p * 64 + lane) >> 1;   // of 16 codes; past K they are zeros
        *reinterpret_cast<uint2*>(xl + tok * KMAX + ((piece ^ (tok & 7)) << 4) + (lane & 1) * 8) = int8_codes8(xv[p], q);
      }
      if (lane == 0) scales[tok] = q.scale;
    }
    wait_lgkm0();
    bare_barrier();
    xsc = scales[t];
#pragma unroll
    for (int i = 0; i < STEPS; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int piece = (wave + i * WAVES) * 8 + 4 * h + g;
        xf[i][h] = *reinterpret_cast<const i32x4*>(xl + t * KMAX + ((piece ^ (t & 7)) << 4));
      }
  }

  i32x4 acc[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] = i32x4{0, 0, 0, 0};
  static_assert(DW == 1 || DW == 2, "one more step may fly");
#pragma unroll
  for (int i = 0; i < STEPS; ++i) {
    if (i + DW <= STEPS) wait_vm<(DW - 1) * 2 * RT>();
    else wait_vm<0>();
    const char* slot = lds + wave * RING + i % DW * (RT * i8::kTileBytes);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const i32x4 wv = *reinterpret_cast<const i32x4*>(slot + rt * i8::kTileBytes + i8::read(r, 4 * h + g));
        acc[rt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xf[i][h], acc[rt], 0, 0, 0);
      }
    if (i + DW < STEPS) {
      wait_lgkm0();   // this step's reads are done before its slot is filled again
      issue(i + DW);
    }
  }

  // the waves' partial tiles, each in its own ring; C lane l holds rows 4*(l/16)+i, token l%16
  wait_lgkm0();
  if (r < a.T) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) *reinterpret_cast<i32x4*>(lds + wave * RING + rt * 1024 + lane * 16) = acc[rt];
  }
  wait_lgkm0();
  bare_barrier();
  static_assert(WAVES >= RT, "a wave for every row tile");
  if (wave < RT && r < a.T && n < a.N) {   // N % 4 == 0: the four rows are in or out together
    i32x4 sum = {0, 0, 0, 0};
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += *reinterpret_cast<const i32x4*>(lds + v * RING + wave * 1024 + lane * 16);
    store4(a.kv + (int64_t)r * a.N + n, sum, xsc, wsc);
  }
}

template <int RT, int WAVES, int DW, int STEPS>
constexpr int reg_lds(bool xbf, int T) {
  return WAVES * DW * RT * i8::kTileBytes + (xbf ? T * (WAVES * STEPS * i8::kStep + 4) : 0);
}

// ---- more tokens, or a longer K: a shared ring of slices ----
//
// A workgroup's waves share slices of 128 k of its 16*RT rows and 16*NT tokens,
// fetched D - 1 slices ahead into a ring of D. Wave (ks, j) multiplies token tile j
// with every row tile, both 64-k halves of a slice (KS 1) or one (KS 2), so that
// little is left to add at the end: with the waves splitting k alone each held every
// tile, and RT * NT * WAVES KiB went through LDS behind the last load (T 61 11.4
// against 9.8 us, T 32 9.5 against 8.5).
//
// Workgroups start at different slices: rows a multiple of some KiB apart that are
// all read at the same k fall on few memory channels (N 28672, K 4096, T 16 / 61:
// 25.9 / 28.4 -> 22.5 / 23.9 us; N 12288: 10.0 / 10.8 -> 9.0 / 10.4).
template <int RT, int NT, int KS>
struct Slice {
  static constexpr int WAVES = NT * KS;
  static constexpr int PER = 2 * (RT + NT);                       // DMAs of a slice
  static constexpr int IPW = (PER + WAVES - 1) / WAVES;           // of a wave; some fill the slot's padding
  static constexpr int SLOT = IPW * WAVES * 1024;
  static constexpr int red = KS * NT * RT * 1024;
  static constexpr int lds(int depth) { return depth * SLOT > red ? depth * SLOT : red; }
  static_assert(KS == 1 || KS == 2, "halves of a slice");
};

template <int RT, int NT, int KS, int D>
__global__ __launch_bounds__(NT * KS * 64) void gemv_int8_slice_kernel(const GemvI8Args a) {
  using S = Slice<RT, NT, KS>;
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int WAVES = S::WAVES, IPW = S::IPW;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int ks = wave / NT, j = wave % NT;
  const int n0 = blockIdx.x * 16 * RT, rows = min(16 * RT, a.N - n0);
  const int t0 = blockIdx.y * 16 * NT, T = min(16 * NT, a.T - t0);
  const int g = lane >> 4, r = lane & 15;
  const uint32_t K = (uint32_t)a.K;
  const rsrc_t rw = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)rows * K);
  const rsrc_t rx = make_rsrc((const uint8_t*)a.x + (int64_t)t0 * a.K, (uint32_t)T * K);
  const int nk = (a.K + i8::kStep - 1) / i8::kStep;

  // what this thread adds up and stores: row tiles ks, ks + KS, .. of token tile j
  constexpr int MINE = (RT + KS - 1) / KS;
  const int t = j * 16 + r;
  f32x4 wsc[MINE];
  const float xsc = t < T ? a.xs[t0 + t] : 0.f;
#pragma unroll
  for (int m = 0; m < MINE; ++m) {
    const int n = n0 + (ks + KS * m) * 16 + 4 * g;
    wsc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (n < a.N) wsc[m] = *reinterpret_cast<const f32x4*>(a.ws + n);
  }

  // DMA q of a slice: 8 rows of W (q < 2 RT) or of x. The slice's offset in the
  // rows is added to a lane's own; kOob sends the whole past both ranges, for a
  // slice that does not exist and for the pieces past the rows' ends.
  uint32_t vofs[IPW];
#pragma unroll
  for (int i = 0; i < IPW; ++i) {
    const int q = wave + WAVES * i;
    vofs[i] = q < S::PER ? i8::voffset(lane, q < 2 * RT ? q : q - 2 * RT, 0u, K) : 0u;
  }
  const bool tail = (uint32_t)(nk - 1) * i8::kStep + i8::piece_of(lane) >= K;
  int at = (int)(blockIdx.x % (uint32_t)nk), left = nk, wslot = 0;
  auto issue = [&]() {
    const uint32_t kofs = left > 0 ? (uint32_t)at * i8::kStep : i8::kOob;
    const uint32_t ko = tail && at == nk - 1 ? i8::kOob : kofs;
#pragma unroll
    for (int i = 0; i < IPW; ++i) {
      const int q = wave + WAVES * i;
      const uint32_t vo = q < S::PER ? vofs[i] + ko : i8::kOob;
      if (q < 2 * RT)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(lds + wslot + q * 1024), 16, vo, 0, 0, 0);
      else
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(lds + wslot + q * 1024), 16, vo, 0, 0, 0);
    }
    at = at + 1 == nk ? 0 : at + 1;
    --left;
    wslot = wslot == (D - 1) * S::SLOT ? 0 : wslot + S::SLOT;
  };
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) issue();

  i32x4 acc[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) acc[rt] = i32x4{0, 0, 0, 0};
  const char* slot = lds;
  for (int d = 0; d < nk; ++d) {
    wait_vm<(D - 2) * IPW>();
    bare_barrier();   // slice d is there; every wave has read slice d-1
    issue();
    auto multiply = [&](int h) {
      const int o = i8::read(r, 4 * h + g);
      const i32x4 xb = *reinterpret_cast<const i32x4*>(slot + (RT + j) * i8::kTileBytes + o);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const i32x4 wv = *reinterpret_cast<const i32x4*>(slot + rt * i8::kTileBytes + o);
        acc[rt] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wv, xb, acc[rt], 0, 0, 0);
      }
    };
    if constexpr (KS == 1) {
      multiply(0);
      multiply(1);
    } else {
      multiply(ks);
    }
    wait_lgkm0();
    slot = slot == lds + (D - 1) * S::SLOT ? lds : slot + S::SLOT;
  }
  wait_vm<0>();   // the last slices' DMAs of zeros: none may land once the wave has ended
  if constexpr (KS > 1) {
    bare_barrier();   // no DMA and no read is left
    i32x4* red = reinterpret_cast<i32x4*>(lds);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) red[((ks * NT + j) * RT + rt) * 64 + lane] = acc[rt];
    wait_lgkm0();
    bare_barrier();
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int rt = ks + KS * m;
      if (rt < RT) {
        i32x4 sum = {0, 0, 0, 0};
#pragma unroll
        for (int v = 0; v < KS; ++v) sum += red[((v * NT + j) * RT + rt) * 64 + lane];
        acc[m] = sum;
      }
    }
  }
  // C lane l holds rows 4*(l/16)+i of the row tile, token l%16
#pragma unroll
  for (int m = 0; m < MINE; ++m) {
    const int rt = ks + KS * m, n = n0 + rt * 16 + 4 * g;
    if (rt < RT && t < T && n < a.N) store4(a.kv + (int64_t)(t0 + t) * a.N + n, acc[m], xsc, wsc[m]);   // N % 4 == 0
  }
}

template <int RT, int WAVES, int DW, int STEPS, bool XBF>
hipError_t reg(const GemvI8Args& a, hipStream_t s) {
  const int lds = reg_lds<RT, WAVES, DW, STEPS>(XBF, a.T);
  const auto fn = gemv_int8_reg_kernel<RT, WAVES, DW, STEPS, XBF>;
  if (reg_lds<RT, WAVES, DW, STEPS>(XBF, 16) > 64 * 1024) {   // above the default limit
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((a.N + 16 * RT - 1) / (16 * RT)), dim3(WAVES * 64), lds, s, a);
  return hipGetLastError();
}

template <int RT, int NT, int KS, int D>
hipError_t slices(const GemvI8Args& a, hipStream_t s) {
  constexpr int lds = Slice<RT, NT, KS>::lds(D);
  const auto fn = gemv_int8_slice_kernel<RT, NT, KS, D>;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((a.N + 16 * RT - 1) / (16 * RT), (a.T + 16 * NT - 1) / (16 * NT)), dim3(NT * KS * 64), lds, s,
                     a);
  return hipGetLastError();
}

// int8 x in registers: one row tile a workgroup, its whole K in flight at once up to
// K 4096 (N 28672, K 4096, T 1: 20.0 us, slices 21.6; N 4096, K 2048: 2.4, slices 3.5).
hipError_t run_reg(const GemvI8Args& a, hipStream_t s) {
  if (a.K <= 512) return reg<1, 4, 1, 1, false>(a, s);
  if (a.K <= 1024) return reg<1, 8, 1, 1, false>(a, s);
  if (a.K <= 2048) return reg<1, 8, 2, 2, false>(a, s);
  if (a.K <= 4096) return reg<1, 16, 2, 2, false>(a, s);
  return a.K <= 6144 ? reg<1, 16, 2, 3, false>(a, s) : reg<1, 16, 2, 4, false>(a, s);
}

// bf16 x: three row tiles where there are many, for each workgroup quantizes x (N
// 20480, K 2048, T 8: 8.1 us, one tile 9.0).
hipError_t run_reg_bf16(const GemvI8Args& a, hipStream_t s) {
  const bool many = (a.N + 15) / 16 > dev_info().num_cus;
  if (a.K <= 512) return reg<1, 4, 1, 1, true>(a, s);
  if (a.K <= 1024) return many ? reg<3, 8, 1, 1, true>(a, s) : reg<1, 8, 1, 1, true>(a, s);
  if (a.K <= 2048) return many ? reg<3, 8, 1, 2, true>(a, s) : reg<1, 8, 2, 2, true>(a, s);
  return many && a.T <= 8 ? reg<3, 16, 1, 2, true>(a, s) : reg<1, 16, 2, 2, true>(a, s);   // LDS holds the codes of T rows
}

// Slices. Up to one row tile for a compute unit: one a workgroup. Up to four: few
// tokens still one (several workgroups on a compute unit), more tokens two or three
// and the slice's halves on two waves. Beyond: smaller rings, more workgroups on a
// compute unit; from 33 tokens on seven row tiles where the compute units then have
// fewer rows in their fullest round (N 28672, T 61: 23.9 us, three 31.6; N 20480
// 10.4, three 9.8). Past 64 tokens six waves, a token tile each, are enough without
// halves.
template <int NT>
hipError_t run_slices(const GemvI8Args& a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, cus = dev_info().num_cus;
  auto rows = [&](int rt) { return ((tiles + rt - 1) / rt + cus - 1) / cus * rt; };
  if constexpr (NT == 1) {
    return tiles <= cus ? slices<1, 1, 2, 4>(a, s) : slices<1, 1, 1, 4>(a, s);
  } else if constexpr (NT == 2) {
    return tiles <= cus ? slices<1, 2, 1, 4>(a, s) : tiles <= 4 * cus ? slices<2, 2, 2, 4>(a, s) : slices<2, 2, 1, 3>(a, s);
  } else if constexpr (NT <= 4) {
    return tiles <= cus        ? slices<1, NT, 1, 4>(a, s)
           : tiles <= 4 * cus  ? slices<3, NT, 2, 4>(a, s)
           : rows(7) < rows(3) ? slices<7, NT, 2, 3>(a, s)
                               : slices<3, NT, 2, 3>(a, s);
  } else {
    return tiles <= cus                               ? slices<1, NT, 1, 3>(a, s)
           : tiles > 4 * cus && rows(7) < rows(3) ? slices<7, NT, 1, 3>(a, s)
                                                      : slices<3, NT, 1, 3>(a, s);
  }
}

// Workgroups of rt row tiles and nt token tiles.
int64_t groups(int64_t T, int N, int rt, int nt) {
  return ((N + 16LL * rt - 1) / (16 * rt)) * ((T + 16LL * nt - 1) / (16 * nt));
}

}  // namespace

// Few tokens: x in registers up to K 8192, from 9 tokens on (16 rows of x to
// fetch for a wave) only where the workgroups are few: N 4096, K 2048, T 16: 3.2 us,
// slices 3.6; N 20480 8.8, slices 8.0. (A grid holds fewer than 2^32 threads, and
// these have up to 1024 for 16 rows: past N 2^24 the slices' 64 take over.)
hipError_t launch_gemv_int8(const uint8_t* xq, const float* xs, int64_t T, int K, const uint8_t* w, const float* ws, int N,
                            void* kv, hipStream_t s) {
  const GemvI8Args a{xq, xs, w, ws, (uint16_t*)kv, (int)T, K, N};
  if (T <= 8 ? K <= 8192 && N <= 1 << 24 : T <= 16 && K <= 4096 && (N + 15) / 16 <= 2 * dev_info().num_cus)
    return run_reg(a, s);
  if (T <= 16) return run_slices<1>(a, s);
  if (T <= 32) return run_slices<2>(a, s);
  if (T <= 48) return run_slices<3>(a, s);
  if (T <= 64) return run_slices<4>(a, s);
  const int cus = dev_info().num_cus;
  if (groups(T, N, 1, 4) <= cus) return slices<1, 4, 1, 4>(a, s);
  if (T <= 96) return run_slices<6>(a, s);
  return groups(T, N, 4, 4) <= cus ? slices<4, 4, 2, 3>(a, s) : slices<3, 8, 1, 3>(a, s);
}

// Past 64 tokens the smallest tiles that a compute unit each is enough for: 16 rows x 64
// tokens, 64 x 64, 48 x 128. The GEMM's 128 x 128 would leave compute units idle (N 1024,
// K 2048, T 200 4.9 us, 128x128 tiles 9.3; N 4096, T 256 6.5 against 9.5; N 6000, T 200 8.4
// against 10.0; T 128 N 1024 4.8, one group of 128 tokens 5.9). From one token tile of
// its own the GEMM has enough of them only where W is long: up to 96 tokens never, up to
// 128 past four row tiles a compute unit (T 128, N 20480, K 2048: 11.2 us, here 13.3).
bool gemv_int8_supported(int64_t T, int N) {
  const int cus = dev_info().num_cus;
  return T >= 1 && (T <= 96 || (T <= 128 && (N + 15) / 16 <= 4 * cus) || groups(T, N, 4, 4) <= cus ||
                    groups(T, N, 3, 8) <= cus);
}

// Quantizing on the way pays while the launch it saves (2.0 to 2.4 us, and 4 of the host's)
// is more than the work that every workgroup repeats: T 8, N 20480, K 2048 8.1 us against
// 10.2, T 16 13.0 against 10.8, N 12288 8.1 against 8.4, N 4096 5.6 against 6.3; K 4096, T
// 16, N 4096 7.6 against 7.9, N 8192 13.0 against 10.6; T 4, N 28672, K 4096 (117 MB of
// weight) 24.9 against 22.6.
bool gemv_int8_bf16_supported(int64_t T, int K, int N) {
  return T >= 1 && (T <= 8 || (T <= 16 && N <= (K <= 2048 ? 12288 : 4096))) && K <= 4096 && (int64_t)N * K <= 64 << 20;
}

hipError_t launch_gemv_int8_bf16(const void* x, int64_t T, int K, const uint8_t* w, const float* ws, int N, void* kv,
                                 hipStream_t s) {
  return run_reg_bf16({x, nullptr, w, ws, (uint16_t*)kv, (int)T, K, N}, s);
}

}  // namespace engram
