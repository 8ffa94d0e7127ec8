// Tiled projection GEMM in 8-bit integers: kv[T, N] = bf16(float(x . W^T) * xs[t]
// * ws[n]), x int8 [T, K] with one fp32 scale a token, W int8 [N, K] with one a
// row, K % 16 == 0, N % 4 == 0.
//
// The sums are whole numbers in 32 bits, exact for K < 2^17 (128 * 128 * K <
// 2^31), so every order of them gives the same kv: tiles, the small-batch
// kernel (gemv_int8.hip) and any split agree bit for bit. Three fp32 roundings
// (the sum to fp32, two scales) and kv's own are left.
//
// v_mfma_i32_32x32x32_i8 takes in lane l (row l%32, half h = l/32) 16 bytes of k,
// and the order of k is free as long as both operands follow it: sub-step kk
// (0..3) of a 128-byte slice is pieces 2kk + h of the rows, the byte layout of
// the bf16 GEMM (gemm.hip) with twice the k in a slice, at the same cycles a
// matrix instruction. So the block (256 x 256, four waves of 128 x 128, or 128 x
// 128 with two workgroups on a compute unit), the ring of five LDS chunks, the
// tile order and the epilogue are that kernel's; the schedule is described
// there.
//
// The scales wait in registers, two of the wave's 128 (64) rows and tokens a
// lane, and go through LDS once the loop has left it.
#include <algorithm>

#include "gemm_tile.h"

namespace engram {

namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// The accumulators as fp32 times their scales, and to kv (store_tile). The wave's
// scales go through its own KiB of LDS past the epilogue's staging tile: 64 * NT
// different ones a lane would be needed at its accumulators. LDS is free.
template <int NT>
__device__ __forceinline__ void scale_and_store(const i32x16 (&acc)[NT][NT], const float (&wsc)[NT / 2],
                                                const float (&xsc)[NT / 2], char* smem, uint16_t* __restrict__ kv, int T,
                                                int N, int t0, int n0, int wn, int wt, int lane, int wave,
                                                const GateEpi& ep) {
  const int lrow = lane & 31, lhalf = lane >> 5;
  float* sl = reinterpret_cast<float*>(smem + 64 * NT * 128 * NT) + wave * 256;
#pragma unroll
  for (int k = 0; k < NT / 2; ++k) {
    sl[64 * k + lane] = wsc[k];
    sl[128 + 64 * k + lane] = xsc[k];
  }
  wait_lgkm0();
  float tx[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) tx[j] = sl[128 + j * 32 + lrow];
  f32x16 out[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      // accumulator r of lane l: row 8*(r/4) + 4*(l/32) + r%4, token l%32
      const f32x4 wv = *reinterpret_cast<const f32x4*>(sl + i * 32 + 8 * g + 4 * lhalf);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) out[i][j][4 * g + e] = (float)acc[i][j][4 * g + e] * tx[j] * wv[e];
    }
  store_tile<NT>(out, smem, kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

struct GemmI8Args {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* w;
  const float* ws;
  uint16_t* kv;
  int T, K, N;
};

// The 64 * NT square tile of workgroup bid.
template <int NT, bool KTAIL>
__device__ __forceinline__ void ring_tile(const GemmI8Args& p, char* smem, int bid, int tiles_n, int tiles_t,
                                          const GateEpi& ep) {
  const uint8_t* __restrict__ xq = p.xq;
  const uint8_t* __restrict__ w = p.w;
  const float* __restrict__ xs = p.xs;
  const float* __restrict__ ws = p.ws;
  const int T = p.T, K = p.K, N = p.N;
  int tn, tt;
  tile_of(bid, tiles_n, tiles_t, tn, tt);
  constexpr int TILE = 64 * NT, CH = Q_ROW * TILE, NDMA = 2 * NT;   // a chunk in LDS, a wave's DMAs for it
  const int n0 = tn * TILE, t0 = tt * TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * (32 * NT), wt = (wave & 1) * (32 * NT);
  const uint32_t row_bytes = (uint32_t)K;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * K, (uint32_t)min(TILE, N - n0) * row_bytes);
  const rsrc_t rb = make_rsrc(xq + (int64_t)t0 * K, (uint32_t)min(TILE, T - t0) * row_bytes);
  const uint32_t oob = (uint32_t)TILE * row_bytes;   // at or past both ranges
  const int nk = (K + Q_ROW - 1) / Q_ROW;

  // scales of the wave's rows and tokens lane and 64 + lane (rows past the end: the last's, never stored)
  float wsc[NT / 2], xsc[NT / 2];
#pragma unroll
  for (int k = 0; k < NT / 2; ++k) {
    wsc[k] = ws[min(n0 + wn + 64 * k + lane, N - 1)];
    xsc[k] = xs[min(t0 + wt + 64 * k + lane, T - 1)];
  }

  const dma::Lane dl = dma::lane_of(wave, lane, row_bytes);
  auto dma = [&](int slot_ofs, int op, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(op ? rb : ra, (lds_ptr_t)(smem + slot_ofs + (wave + 4 * i) * 1024), 16,
                                             dma::voffset(dl, i, kofs, row_bytes, oob, KTAIL), 0, 0, 0);
  };

  i32x16 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int lrow = lane & 31, lhalf = lane >> 5;
  const int fsw = (lrow >> 1) & 7;
  i32x4 a[2][NT], b[2][NT];
  // fragment f (b of each token block, then a of each row block) of sub-step kk into register set c
  auto frag = [&](int sa, int sb, int kk, int c, int f) {
    const int i = f % NT;
    const int row = (f < NT ? wt : wn) + i * 32 + lrow;
    const int piece = (2 * kk + lhalf) ^ fsw;
    const i32x4 v = *reinterpret_cast<const i32x4*>(smem + (f < NT ? sb : sa) + row * Q_ROW + piece * 16);
    if (f < NT) b[c][i] = v; else a[c][i] = v;
  };
  auto mfma_row = [&](int c, int i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[c][i], b[c][j], acc[i][j], 0, 0, 0);
  };

  // prologue: A0 -> slot 0, B0 -> slot 1, A1 -> slot 2
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(0, 0, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(CH, 1, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(2 * CH, 0, nk > 1 ? (uint32_t)Q_ROW : oob, i);
  wait_vm<NDMA>();
  // a use here keeps the scale loads ahead of the DMAs
#pragma unroll
  for (int k = 0; k < NT / 2; ++k) asm volatile("" : "+v"(wsc[k]), "+v"(xsc[k]));
  bare_barrier();
#pragma unroll
  for (int f = 0; f < 2 * NT; ++f) frag(0, CH, 0, 0, f);

  // Chunk c (A_d = 2d, B_d = 2d+1) lives in ring slot c % 5. While slice d is
  // computed, B_{d+1} and A_{d+2} are fetched into the slots of A_{d-1} and
  // B_{d-1}, freed by the previous slice's barrier.
  int base = 0;   // (2d) % 5
  for (int d = 0; d < nk; ++d) {
    auto slot = [&](int m) { const int v = base + m; return (v >= Q_SLOTS ? v - Q_SLOTS : v) * CH; };
    const int sa = slot(0), sb = slot(1), sa1 = slot(2), sb1 = slot(3), sa2 = slot(4);
    const uint32_t kb1 = d + 1 < nk ? (uint32_t)(d + 1) * Q_ROW : oob;
    const uint32_t ka2 = d + 2 < nk ? (uint32_t)(d + 2) * Q_ROW : oob;
    // sub-step 0: MFMAs on set 0; sub-step 1's fragments into set 1; B_{d+1}
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      dma(sb1, 1, kb1, 2 * q);
      dma(sb1, 1, kb1, 2 * q + 1);
      frag(sa, sb, 1, 1, 2 * q);
      frag(sa, sb, 1, 1, 2 * q + 1);
      mfma_row(0, q);
      SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
      if (NT == 4) { SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); }
      else { SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); }
    }
    // sub-steps 1 and 2: A_{d+2}
#pragma unroll
    for (int kk = 1; kk < 3; ++kk) {
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        __builtin_amdgcn_sched_barrier(0);
        dma(sa2, 0, ka2, (kk - 1) * NT + q);
        frag(sa, sb, kk + 1, (kk + 1) & 1, 2 * q);
        frag(sa, sb, kk + 1, (kk + 1) & 1, 2 * q + 1);
        mfma_row(kk & 1, q);
        if (NT == 4) {
          SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1);
          SGB(SG_MFMA, 1);
        } else {
          SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 1);
        }
      }
    }
    // sub-step 3, first row block, then publish slice d+1: only A_{d+2}'s DMAs may still fly
    __builtin_amdgcn_sched_barrier(0);
    mfma_row(1, 0);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<NDMA>();
    wait_lgkm0();
    bare_barrier();
    // the other row blocks: slice d+1's sub-step-0 fragments into set 0
#pragma unroll
    for (int q = 1; q < NT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      const int f0 = NT == 2 ? 0 : 3 * (q - 1), nf = NT == 2 ? 4 : q == 3 ? 2 : 3;
#pragma unroll
      for (int f = 0; f < nf; ++f) frag(sa1, sb1, 0, 0, f0 + f);
      mfma_row(1, q);
      if (NT == 2) {
        SGB(SG_MFMA, 1); SGB(SG_DSR, 4); SGB(SG_MFMA, 1);
      } else if (q < 3) {
        SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1);
        SGB(SG_MFMA, 1);
      } else {
        SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 2);
      }
    }
    base = base + 2 >= Q_SLOTS ? base + 2 - Q_SLOTS : base + 2;
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  wait_lgkm0();
  bare_barrier();

  scale_and_store<NT>(acc, wsc, xsc, smem, p.kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

// 128x128 tiles where there are at most as many as compute units: nothing else covers a
// late slice there, so all of LDS is one ring of five slices (A and B, 32 KiB), fetched
// four ahead, and the workgroups start at different slices (rows some KiB apart that
// are all read at the same k fall on few memory channels; the order of k is free).
// K 8192, N 8192, T 180 36.0 -> 26.0 us; K 4096, N 12288, T 180 21.1 -> 17.1, N 16384, T
// 256 27.7 -> 20.5; K 2048, N 20480, T 128 12.9 -> 11.2. What is left is LDS: a wave's 64
// x 64 reads 64 KiB a slice and workgroup, its DMAs write 32, at 128 bytes a clock more
// than its 512 clocks of matrix instructions. (256 x 128 with three quarters of that a
// product, three slices in the ring: as fast as two 128x128 workgroups on a compute unit
// within 3%, 7% faster where it just fills a round; not taken.)
constexpr int kDeep = 5;

// The 128x128 tile of workgroup bid, tile columns from tn0 on.
template <bool KTAIL>
__device__ __forceinline__ void deep_tile(const GemmI8Args& p, char* smem, int bid, int tn0, int tiles_n, int tiles_t) {
  const uint8_t* __restrict__ xq = p.xq;
  const uint8_t* __restrict__ w = p.w;
  const float* __restrict__ xs = p.xs;
  const float* __restrict__ ws = p.ws;
  const int T = p.T, K = p.K, N = p.N;
  int tn, tt;
  tile_of(bid, tiles_n, tiles_t, tn, tt);
  constexpr int NT = 2, TILE = 128, CH = Q_ROW * TILE, SLOT = 2 * CH, NDMA = 4;   // of an operand and wave
  const int n0 = (tn0 + tn) * TILE, t0 = tt * TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * 64, wt = (wave & 1) * 64;
  const uint32_t row_bytes = (uint32_t)K;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * K, (uint32_t)min(TILE, N - n0) * row_bytes);
  const rsrc_t rb = make_rsrc(xq + (int64_t)t0 * K, (uint32_t)min(TILE, T - t0) * row_bytes);
  const uint32_t oob = (uint32_t)TILE * row_bytes;   // at or past both ranges
  const int nk = (K + Q_ROW - 1) / Q_ROW;
  float wsc[1] = {ws[min(n0 + wn + lane, N - 1)]}, xsc[1] = {xs[min(t0 + wt + lane, T - 1)]};

  const dma::Lane dl = dma::lane_of(wave, lane, row_bytes);
  int at = tn % nk, left = nk, wslot = 0;      // the slice to fetch next, and its slot
  auto fetch = [&](int i) {                    // DMA i of A (0..3), then of B
    const uint32_t kofs = left > 0 ? (uint32_t)at * Q_ROW : oob;
    const int q = i & 3;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(i < NDMA ? ra : rb,
                                             (lds_ptr_t)(smem + wslot + (i < NDMA ? 0 : CH) + (wave + 4 * q) * 1024), 16,
                                             dma::voffset(dl, q, kofs, row_bytes, oob, KTAIL), 0, 0, 0);
  };
  auto fetched = [&]() {
    at = at + 1 == nk ? 0 : at + 1;
    --left;
    wslot = wslot == (kDeep - 1) * SLOT ? 0 : wslot + SLOT;
  };

  i32x16 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  const int lrow = lane & 31, lhalf = lane >> 5;
  const int fsw = (lrow >> 1) & 7;
  i32x4 a[2][NT], b[2][NT];
  auto frags = [&](int slot, int kk, int c) {
    const int piece = ((2 * kk + lhalf) ^ fsw) * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      b[c][i] = *reinterpret_cast<const i32x4*>(smem + slot + CH + (wt + i * 32 + lrow) * Q_ROW + piece);
      a[c][i] = *reinterpret_cast<const i32x4*>(smem + slot + (wn + i * 32 + lrow) * Q_ROW + piece);
    }
  };
  auto mfma_row = [&](int c, int i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(a[c][i], b[c][j], acc[i][j], 0, 0, 0);
  };

  __builtin_amdgcn_sched_barrier(0);   // the scale loads first
#pragma unroll
  for (int d = 0; d < kDeep - 1; ++d) {
#pragma unroll
    for (int i = 0; i < 2 * NDMA; ++i) fetch(i);
    fetched();
  }
  wait_vm<(kDeep - 2) * 2 * NDMA>();
  asm volatile("" : "+v"(wsc[0]), "+v"(xsc[0]));
  bare_barrier();
  frags(0, 0, 0);
  int slot = 0;
  for (int d = 0; d < nk; ++d) {
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 3 * kk; i < (kk == 2 ? 8 : 3 * kk + 3); ++i) fetch(i);
      frags(slot, kk + 1, (kk + 1) & 1);
      mfma_row(kk & 1, 0);
      mfma_row(kk & 1, 1);
      SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
      SGB(SG_MFMA, 1);
      if (kk < 2) SGB(SG_VMEM, 1);
      SGB(SG_DSR, 2); SGB(SG_MFMA, 1);
    }
    fetched();
    const int next = slot == (kDeep - 1) * SLOT ? 0 : slot + SLOT;
    __builtin_amdgcn_sched_barrier(0);
    mfma_row(1, 0);
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<(kDeep - 2) * 2 * NDMA>();   // slice d+1 is there
    wait_lgkm0();
    bare_barrier();
    __builtin_amdgcn_sched_barrier(0);
    frags(next, 0, 0);
    mfma_row(1, 1);
    SGB(SG_MFMA, 1); SGB(SG_DSR, 4); SGB(SG_MFMA, 1);
    slot = next;
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  wait_lgkm0();
  bare_barrier();
  scale_and_store<NT>(acc, wsc, xsc, smem, p.kv, T, N, t0, n0, wn, wt, lane, wave, GateEpi{});
}

// Two 128x128 workgroups on a compute unit that run in step load at the same time,
// multiply at the same time and store at the same time; over several rounds they may
// stay so. The second one of the first round (workgroups cus .. 2 cus - 1, as they are
// handed out one to a compute unit, then another; only time rests on that) therefore
// starts `pause` * 256 clocks late: 5 for each slice of a tile, at most 25, about the 3 us
// a tile takes outside its loop. That much whatever the K above 640 (us without / 12 / 25 /
// 40 / 60): N 19828, K 640, T 3388 81 / 80 / 72 / 79 / 84, N 11932, K 928, T 4299 84 / 84 / 80 /
// 80 / 86, N 15876, K 1120, T 2687 80 / 78 / 73 / 73 / 79; from K 1680 on none of them is 3%
// from another (N 7380, K 1872, T 2861 60.5 / 60.1 / 60.4 / 60.3 / 60.0). Shorter K: N 4264,
// K 448, T 5058 24.8 -> 21 - 22. Without it the same launch may take half as long again (N
// 10240, K 512, T 3000 27 or 49, with it 26 - 28). A launch of one round gains nothing.
template <int NT, bool KTAIL>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(NT == 4 ? 1 : 2, NT == 4 ? 1 : 2)))
void gemm_int8_kernel(const GemmI8Args p, int tiles_n, int tiles_t, uint32_t cus, int pause, GateEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  if (NT == 2 && blockIdx.x - cus < cus)
    for (int i = 0; i < pause; ++i) __builtin_amdgcn_s_sleep(4);
  ring_tile<NT, KTAIL>(p, smem, blockIdx.x, tiles_n, tiles_t, ep);
}

template <bool KTAIL>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_int8_deep_kernel(const GemmI8Args p, int tiles_n, int tiles_t) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  deep_tile<KTAIL>(p, smem, blockIdx.x, 0, tiles_n, tiles_t);
}

// Whole rounds of 256x256 tiles (`big` columns of them), then 128x128 ones on the
// compute units as they come free. One launch: N 20480, K 4096, T 1000 (256 + 256 tiles)
// 76 us, two launches 79 - 81; N 12288, K 4096, T 2048 91 against 92. The small tiles
// have all of LDS here and so take the deep ring; two in half of it each, in a launch of
// their own, are 1.5% faster at best (N 28672, K 2048, T 700 46.6 against 47.3).
template <bool KTAIL>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_int8_mixed_kernel(const GemmI8Args p, int big) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  const int tiles_t = (p.T + 255) / 256, first = big * tiles_t, bid = blockIdx.x;
  if (bid < first)
    ring_tile<4, KTAIL>(p, smem, bid, big, tiles_t, GateEpi{});
  else
    deep_tile<KTAIL>(p, smem, bid - first, 2 * big, (p.N + 127) / 128 - 2 * big, (p.T + 127) / 128);
}

template <typename F, typename... A>
hipError_t launch_gemm(F fn, int64_t grid, int lds, hipStream_t s, const A&... args) {
  const hipError_t e = set_lds((const void*)fn, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3((uint32_t)grid), dim3(THREADS), lds, s, args...);
  return hipGetLastError();
}

constexpr int kDeepLds = kDeep * 2 * 128 * Q_ROW;
static_assert(kDeepLds <= Q_LDS, "one workgroup's LDS");

template <int NT>
hipError_t launch_ring(const GemmI8Args& p, hipStream_t s, const GateEpi& ep) {
  const int tiles_n = (p.N + 64 * NT - 1) / (64 * NT), tiles_t = (p.T + 64 * NT - 1) / (64 * NT);
  const int64_t tiles = (int64_t)tiles_n * tiles_t, cus = dev_info().num_cus;
  const int pause = tiles > 2 * cus ? std::min(25, 5 * ((p.K + Q_ROW - 1) / Q_ROW)) : 0;
  return launch_gemm(p.K % Q_ROW ? gemm_int8_kernel<NT, true> : gemm_int8_kernel<NT, false>, tiles, Q_LDS * NT / 4, s, p,
                     tiles_n, tiles_t, (uint32_t)cus, pause, ep);
}

hipError_t launch_deep(const GemmI8Args& p, hipStream_t s) {
  const int tiles_n = (p.N + 127) / 128, tiles_t = (p.T + 127) / 128;
  return launch_gemm(p.K % Q_ROW ? gemm_int8_deep_kernel<true> : gemm_int8_deep_kernel<false>, (int64_t)tiles_n * tiles_t,
                     kDeepLds, s, p, tiles_n, tiles_t);
}

hipError_t launch_mixed(const GemmI8Args& p, int big, hipStream_t s) {
  const int64_t grid = (int64_t)big * ((p.T + 255) / 256) + (int64_t)((p.N + 127) / 128 - 2 * big) * ((p.T + 127) / 128);
  return launch_gemm(p.K % Q_ROW ? gemm_int8_mixed_kernel<true> : gemm_int8_mixed_kernel<false>, grid, Q_LDS, s, p, big);
}

}  // namespace

// At most one 128x128 tile for a compute unit and enough slices that their latency
// counts (K 2048, N 4096, T 180: nothing gained). Of one tile of
// tokens, where the weight streams from HBM, three quarters as many (T 128, N 28672, K
// 4096: 24.1 us, deep 28.4).
static bool int8_deep(int64_t T, int64_t N, int K) {
  const int64_t tiles = ((N + 127) / 128) * ((T + 127) / 128), cus = dev_info().num_cus;
  return 4 * tiles <= (T <= 128 ? 3 : 4) * cus && (K >= 4096 || (K >= 2048 && 2 * tiles > cus));
}

// The other GEMMs' model (gemm_tile.h) with times of this one's. It charges the split
// as two launches with two 128x128 tiles on a compute unit; here it is one launch and
// they run one on a compute unit, in the deep ring. The times are fitted to what is
// launched, the charge keeps the split to where it surely pays: N 6588, K 4000, T 4955
// 128x128 tiles 166 us, split 143; N 10924, K 2240, T 1764 59 and 55; the other way N
// 11932, K 928, T 4299 80 and 84.
static int int8_big_columns(int64_t T, int N, int K) {
  return big_columns(T, N, (K + 127) / 128 * 128, {9000, 1430, 3300, 870, 3200, 660});
}

bool gemm_int8_big_tiles(int64_t T, int N, int K) { return int8_big_columns(T, N, K) == (N + 255) / 256; }

// The gate's epilogue has the 256x256 tile only.
hipError_t launch_gemm_int8(const uint8_t* xq, const float* xs, int64_t T, int K, const uint8_t* w, const float* ws,
                            int N, void* kv, hipStream_t s, const GateEpi& ep) {
  const GemmI8Args p{xq, xs, w, ws, (uint16_t*)kv, (int)T, K, N};
  if (!ep.hidden && int8_deep(T, N, K)) return launch_deep(p, s);
  const int tn = (N + 255) / 256, big = ep.hidden ? tn : int8_big_columns(T, N, K);   // of 256x256 tiles
  return big == tn ? launch_ring<4>(p, s, ep) : big ? launch_mixed(p, big, s) : launch_ring<2>(p, s, ep);
}

}  // namespace engram
