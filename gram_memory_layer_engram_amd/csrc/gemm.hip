// wkv projection, tiled GEMM for prefill: kv[T, N] = bf16(x[T, K] . W[N, K]^T)
// with bf16 weights (v_mfma_f32_32x32x16_bf16) or MXFP8 weights and MXFP8
// activations (v_mfma_scale_f32_32x32x64_f8f6f4).
//
// "vllm.models.deepseek_v4_1.common.engram", Engram.__init__ / forward: wkv
// is a bias-free linear from n_hash_cols*head_dim (K) to dim*(hc_mult+1) (N)
// on the flattened staged rows. MXFP8 weight format: "vllm.models.
// deepseek_v41.amd.mono.attention.gemv", module docstring (row-major e4m3
// W[N, K], E8M0 byte per 32x32 block S[N/32, K/32]).
//
// MI355X design
//  * Both operands are K-contiguous. A = W rows (n), B = x rows (tokens): an
//    accumulator lane then holds 4 consecutive n of one token.
//  * Block tile 256 (n) x 256 (tokens); four waves in 2x2, each 128x128 =
//    4x4 MFMA tiles of 32x32 (256 fp32 accumulators per lane, in AGPRs). That
//    is the largest tile one CU's register file holds, and at K = 2048 the
//    kernel is bound by L2 -> CU operand traffic (one 256x256 tile reads 2 x
//    256 rows per k) and by the clock the chip sustains with MFMA and that
//    traffic both running, not by MFMA issue: the loop is paced for the
//    address unit, not for the matrix cores.
//  * Global -> LDS with buffer_load ... lds (16 bytes per lane, written at
//    LDS base + lane*16): no staging registers, no ds_write, and the buffer
//    descriptor's range check returns zeros past the last row of W or x, so
//    ragged tiles need no branches; a stage that does not exist is loaded
//    from an offset past the range (zeros into a buffer nobody reads), which
//    keeps the loop free of branches. The range check covers the vector
//    offset only, so every DMA offset (row, k slice, piece) is carried in it
//    and the scalar offset is 0 (gemm_dma.h; a host model of those offsets
//    checks each against the range).
//  * bf16: a k slice is 64 elements, so one DMA instruction fetches 8 rows x
//    128 bytes, 8 whole cache lines (with 32-element stages it touched half
//    of 16 lines: 627 -> 564 us for the prefill GEMM, same instructions,
//    same bytes). LDS rows are 128 bytes of 8 pieces, piece p of row r at
//    p ^ ((r >> 1) & 7), conflict-free for the 32-row fragment reads. Each
//    operand's slice is a 32 KiB chunk in a ring of five (160 KiB, all of
//    LDS): during slice d, B of slice d+1 is fetched first (one DMA per 2
//    MFMAs), then A of slice d+2 (one per 4), so every DMA has at least ~38
//    MFMAs before the barrier that needs it (32 already suffice: a
//    three-stage ring times like a four-stage one). The barrier that
//    publishes slice d+1 sits after the first 4 of the last 16 MFMAs of
//    slice d, and the next slice's first fragments are read under the other
//    12.
//  * MXFP8: the same ring of five 32 KiB chunks, a slice being 128 e4m3 per
//    row (gemm_mx_ring_kernel, described above it), or of five 16 KiB chunks
//    for 128x128 tiles, two workgroups on a compute unit.
//  * Epilogue: the bf16 tile is staged in LDS as [token][n] (512-byte rows,
//    16-byte chunks XOR-swizzled by token) and written back as whole rows,
//    16 bytes per lane: 8 full cache lines per store instruction instead of
//    32 partial ones, which halves the epilogue.
//  * Tile order is XCD-aware (workgroup ids are dealt round-robin over the 8
//    XCDs): ids are regrouped per XCD, then walked in groups of 4 token tiles
//    so the 32 workgroups an XCD runs at once share 4 x-tiles and 8 W-tiles
//    in its L2.
//  * MXFP8: gfx950's 32x32x64 scaled MFMA takes, in lane l (row l%32, group
//    g = l/32), k bytes 16g..16g+15 and 32+16g..32+16g+15 of its 64-k step,
//    and lane group g's E8M0 byte scales k block [32g, 32g+32) (measured on
//    the hardware). Each lane therefore reads pieces 4s+g and 4s+2+g of the
//    stage for sub-step s and passes byte 2s+g of the stage's 4 scale bytes.
#include <type_traits>

#include "gemm_tile.h"

namespace engram {

namespace {

// bf16 wkv GEMM (see the file comment). KTAIL: K % 64 != 0, the last slice's
// pieces past the row end are loaded from past the range (zeros).
template <bool KTAIL>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(1, 1)))
void gemm_bf16_kernel(const uint16_t* __restrict__ x, int T, int K, const uint16_t* __restrict__ w,
                      int N, uint16_t* __restrict__ kv, int tiles_n, int tiles_t, GateEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int tn, tt;
  tile_of(blockIdx.x, tiles_n, tiles_t, tn, tt);
  const int n0 = tn * BM, t0 = tt * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * 128, wt = (wave & 1) * 128;
  const uint32_t row_bytes = (uint32_t)K * 2u;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * K, (uint32_t)min(BM, N - n0) * row_bytes);
  const rsrc_t rb = make_rsrc(x + (int64_t)t0 * K, (uint32_t)min(BN, T - t0) * row_bytes);
  const uint32_t oob = (uint32_t)BM * row_bytes;   // at or past both ranges
  const int nk = (K + 63) / 64;

  // DMA i (0..7) of a chunk: LDS rows 8*(wave + 4i) .. +8 (gemm_dma.h). The
  // whole offset, row step and k offset included, is the range-checked
  // vector offset; the scalar offset stays 0.
  const dma::Lane dl = dma::lane_of(wave, lane, row_bytes);
  auto dma = [&](int slot_ofs, int op, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(op ? rb : ra, (lds_ptr_t)(smem + slot_ofs + (wave + 4 * i) * 1024),
                                             16, dma::voffset(dl, i, kofs, row_bytes, oob, KTAIL), 0, 0, 0);
  };

  f32x16 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  const int lrow = lane & 31, lhalf = lane >> 5;
  const int fsw = (lrow >> 1) & 7;
  bf16x8_t a[2][4], b[2][4];
  // fragment f (0..3: b0..b3, 4..7: a0..a3) of sub-step kk (0..3) into register set c
  auto frag = [&](int sa, int sb, int kk, int c, int f) {
    const int i = f & 3;
    const int row = (f < 4 ? wt : wn) + i * 32 + lrow;
    const int piece = (2 * kk + lhalf) ^ fsw;
    const bf16x8_t v = *reinterpret_cast<const bf16x8_t*>(smem + (f < 4 ? sb : sa) + row * Q_ROW + piece * 16);
    if (f < 4) b[c][i] = v; else a[c][i] = v;
  };
  auto mfma_row = [&](int c, int i) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[c][i], b[c][j], acc[i][j], 0, 0, 0);
  };

  // prologue: A0 -> slot 0, B0 -> slot 1, A1 -> slot 2
#pragma unroll
  for (int i = 0; i < Q_DMA; ++i) dma(0, 0, 0u, i);
#pragma unroll
  for (int i = 0; i < Q_DMA; ++i) dma(Q_CHUNK, 1, 0u, i);
#pragma unroll
  for (int i = 0; i < Q_DMA; ++i) dma(2 * Q_CHUNK, 0, nk > 1 ? (uint32_t)Q_ROW : oob, i);
  wait_vm<Q_DMA>();
  bare_barrier();
#pragma unroll
  for (int f = 0; f < 8; ++f) frag(0, Q_CHUNK, 0, 0, f);

  // Chunk c (A_d = 2d, B_d = 2d+1) lives in ring slot c % 5. While slice d
  // is computed, B_{d+1} (slot (2d+3) % 5) and A_{d+2} (slot (2d+4) % 5) are
  // fetched into the slots of A_{d-1} and B_{d-1}, freed by the previous
  // slice's barrier. The slot offsets are computed per slice (an unrolled
  // ring makes every fragment address loop-invariant: 232 spilled VGPRs).
  int base = 0;   // (2d) % 5
  for (int d = 0; d < nk; ++d) {
    {
      auto slot = [&](int m) { const int v = base + m; return (v >= Q_SLOTS ? v - Q_SLOTS : v) * Q_CHUNK; };
      const int sa = slot(0), sb = slot(1), sa1 = slot(2), sb1 = slot(3), sa2 = slot(4);
      const uint32_t kb1 = d + 1 < nk ? (uint32_t)(d + 1) * Q_ROW : oob;
      const uint32_t ka2 = d + 2 < nk ? (uint32_t)(d + 2) * Q_ROW : oob;
      // sub-step 0: MFMAs on set 0; sub-step 1's fragments into set 1; B_{d+1}, two DMAs per quarter
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        __builtin_amdgcn_sched_barrier(0);
        dma(sb1, 1, kb1, 2 * q);
        dma(sb1, 1, kb1, 2 * q + 1);
        frag(sa, sb, 1, 1, 2 * q);
        frag(sa, sb, 1, 1, 2 * q + 1);
        mfma_row(0, q);
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1);
        SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1);
      }
      // sub-steps 1 and 2: A_{d+2}, one DMA per quarter
#pragma unroll
      for (int kk = 1; kk < 3; ++kk) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          __builtin_amdgcn_sched_barrier(0);
          dma(sa2, 0, ka2, (kk - 1) * 4 + q);
          frag(sa, sb, kk + 1, (kk + 1) & 1, 2 * q);
          frag(sa, sb, kk + 1, (kk + 1) & 1, 2 * q + 1);
          mfma_row(kk & 1, q);
          SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1);
          SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1);
        }
      }
      // sub-step 3, first quarter, then publish slice d+1: each wave waits
      // for its own DMAs of A_{d+1} and B_{d+1} (only A_{d+2}'s 8 may still
      // fly) and for its LDS reads of slice d, then the barrier
      __builtin_amdgcn_sched_barrier(0);
      mfma_row(1, 0);
      __builtin_amdgcn_sched_barrier(0);
      wait_vm<Q_DMA>();
      wait_lgkm0();
      bare_barrier();
      // quarters 1-3: slice d+1's sub-step-0 fragments into set 0 (3 + 3 + 2)
#pragma unroll
      for (int q = 1; q < 4; ++q) {
        __builtin_amdgcn_sched_barrier(0);
        const int f0 = q == 1 ? 0 : (q == 2 ? 3 : 6), nf = q == 3 ? 2 : 3;
#pragma unroll
        for (int f = 0; f < nf; ++f) frag(sa1, sb1, 0, 0, f0 + f);
        mfma_row(1, q);
        if (q < 3) {
          SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1);
          SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1);
        } else {
          SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 2);
        }
      }
    }
    base = base + 2 >= Q_SLOTS ? base + 2 - Q_SLOTS : base + 2;
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  store_tile(acc, smem, kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

constexpr int S_ROW = 128;                      // MXFP8 ring: 128-byte slices (two k steps)

// MXFP8 GEMM on the bf16 kernel's ring. A slice is 128
// e4m3 per row, two MFMA k steps ("stages", 16 MFMAs per wave each), so a
// DMA instruction fetches 8 rows x 128 bytes, 8 whole cache lines. Each
// operand's slice is a 32 KiB chunk in a ring of five (all 160 KiB of LDS),
// chunk c in slot c % 5 with A_d = chunk 2d and B_d = chunk 2d+1. During
// slice d, B_{d+1} goes out in stage 0 (two DMAs per quarter) and A_{d+2} in
// stage 1 (3, 3, 2), into the slots of A_{d-1} and B_{d-1}; the barrier that
// publishes slice d+1 sits after three of stage 1's four MFMA row blocks.
// A's DMAs thus get more than a slice of lead (two 64 KiB slice buffers
// gave every DMA about 37% of one: long-prefill GEMM 3.32 -> 3.16 ms).
// With LDS full, the E8M0 bytes are read from memory into registers, one
// group of four stages (8 bytes per row) ahead, issued at the start of a
// group's first slice, before its DMAs, so the barrier's wait covers them.
// Lane (row l%32, group g = l/32) reads, for stage h, pieces 4h+g and
// 4h+2+g of its row and passes the E8M0 byte of k block 2*stage + g. The
// fragments stream one A row block ahead (two register sets); B and the
// next stage's first A block are read under a stage's last four MFMAs.
// Slices go in pairs; HALF (K % 256 == 128): one more behind the loop, whose
// group of scale bytes is half the row's, half the next row's or zeros, unused.
// NT 4: the 256x256 tile; 2: 128x128, two workgroups on a compute unit.
template <int NT, bool HALF>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(NT == 4 ? 1 : 2, NT == 4 ? 1 : 2)))
void gemm_mx_ring_kernel(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs, int T, int K,
                         const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws, int N,
                         uint16_t* __restrict__ kv, int tn0, int tiles_n, int tiles_t, GateEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int tn, tt;
  tile_of(blockIdx.x, tiles_n, tiles_t, tn, tt);
  constexpr int TILE = 64 * NT, CH = S_ROW * TILE, NDMA = 2 * NT;   // a chunk in LDS, a wave's DMAs for it
  const int n0 = (tn0 + tn) * TILE, t0 = tt * TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * (32 * NT), wt = (wave & 1) * (32 * NT);
  const uint32_t row_bytes = (uint32_t)K;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * K, (uint32_t)min(TILE, N - n0) * row_bytes);
  const rsrc_t rb = make_rsrc(xq + (int64_t)t0 * K, (uint32_t)min(TILE, T - t0) * row_bytes);
  const uint32_t oob = (uint32_t)TILE * row_bytes;   // at or past both ranges
  const int ns = K / 128;                           // slices, odd where HALF
  const int kb = K / 32;                            // scale bytes per row
  const int lrow = lane & 31, lg = lane >> 5;

  const dma::Lane dl = dma::lane_of(wave, lane, row_bytes);
  auto dma = [&](int slot_ofs, int op, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(op ? rb : ra, (lds_ptr_t)(smem + slot_ofs + (wave + 4 * i) * 1024),
                                             16, dma::voffset(dl, i, kofs, row_bytes, oob, false), 0, 0, 0);
  };

  // The 8 scale bytes of stages s4 .. s4+3 (s4 % 4 == 0) of each row, as
  // range-checked vector loads: a scalar load would be waited for by the
  // next fragment read's lgkmcnt(0). Token rows past T read zeros.
  const rsrc_t rsa = make_rsrc(ws, (uint32_t)(N / 32) * (uint32_t)kb);
  const rsrc_t rsb = make_rsrc(xs + (int64_t)t0 * kb, (uint32_t)min(TILE, T - t0) * (uint32_t)kb);
  uint32_t arow[NT], brow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    arow[i] = (uint32_t)min((n0 + wn + i * 32) / 32, N / 32 - 1) * (uint32_t)kb;
    brow[i] = (uint32_t)(wt + i * 32 + lrow) * (uint32_t)kb;
  }
  auto scales8 = [&](int s4, u32x2 (&a8)[NT], u32x2 (&b8)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a8[i] = __builtin_amdgcn_raw_buffer_load_b64(rsa, arow[i] + 2u * (uint32_t)s4, 0, 0);
      b8[i] = __builtin_amdgcn_raw_buffer_load_b64(rsb, brow[i] + 2u * (uint32_t)s4, 0, 0);
    }
  };
  const uint32_t lsh = (uint32_t)lg * 8u;
  auto pick = [&](const u32x2& v, int u) {   // u static: byte 2u + lg
    return (int)(((u < 2 ? v.x : v.y) >> ((uint32_t)(16 * (u & 1)) + lsh)) & 0xffu);
  };
  auto frag = [&](int slot_ofs, int half, int row) {
    const char* base = smem + slot_ofs + row * S_ROW;
    const int sw = (row >> 1) & 7;
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + (((4 * half + lg) ^ sw) << 4));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + (((4 * half + 2 + lg) ^ sw) << 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x16 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  i32x8 a0, a1, b[NT], nb[NT];
  int sa[NT], sb[NT];
  auto mfma_row = [&](const i32x8& a, int i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b[j], acc[i][j], 0, 0, 0, sa[i], 0,
                                                                 sb[j]);
  };

  // prologue: the first group's scale bytes, then A_0 -> slot 0, B_0 -> slot
  // 1, A_1 -> slot 2; wait for all but A_1's DMAs
  u32x2 sa8[NT], sb8[NT], na8[NT], nb8[NT];
  scales8(0, sa8, sb8);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(0, 0, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(CH, 1, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma(2 * CH, 0, ns > 1 ? (uint32_t)S_ROW : oob, i);
  wait_vm<NDMA>();
  // a use here keeps the first group's scale loads ahead of the DMAs (left
  // to itself, the compiler sinks them to the loop, and the waits it then
  // places at the loop head drain every slice's DMAs)
#pragma unroll
  for (int i = 0; i < NT; ++i) asm volatile("" : "+v"(sa8[i]), "+v"(sb8[i]));
  bare_barrier();
#pragma unroll
  for (int j = 0; j < NT; ++j) b[j] = frag(CH, 0, wt + j * 32 + lrow);
  a0 = frag(0, 0, wn + lrow);

  int base = 0;   // (2d) % 5
  // one slice; PAR = d % 2 (the slice's place in its group of two)
  auto slice = [&](int d, auto par) {
    constexpr int PAR = decltype(par)::value;
    auto slot = [&](int m) { const int v = base + m; return (v >= Q_SLOTS ? v - Q_SLOTS : v) * CH; };
    const int s_a = slot(0), s_b = slot(1), s_a1 = slot(2), s_b1 = slot(3), s_a2 = slot(4);
    const uint32_t kb1 = d + 1 < ns ? (uint32_t)(d + 1) * S_ROW : oob;
    const uint32_t ka2 = d + 2 < ns ? (uint32_t)(d + 2) * S_ROW : oob;
    if (PAR == 0) scales8(min(2 * d + 4, 2 * ns - (HALF ? 2 : 4)), na8, nb8);   // the last group reloads itself, unused
    // stage 0: B_{d+1}, two DMAs per quarter
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      sa[i] = pick(sa8[i], 2 * PAR);
      sb[i] = pick(sb8[i], 2 * PAR);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      dma(s_b1, 1, kb1, 2 * q);
      dma(s_b1, 1, kb1, 2 * q + 1);
      if (q < NT - 1) {
        if (q & 1) a0 = frag(s_a, 0, wn + (q + 1) * 32 + lrow);
        else a1 = frag(s_a, 0, wn + (q + 1) * 32 + lrow);
        mfma_row((q & 1) ? a1 : a0, q);
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
        if (NT == 4) SGB(SG_MFMA, 2);
      } else {
#pragma unroll
        for (int j = 0; j < NT; ++j) nb[j] = frag(s_b, 1, wt + j * 32 + lrow);
        a0 = frag(s_a, 1, wn + lrow);
        mfma_row(a1, NT - 1);
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 4); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1);
        if (NT == 4) { SGB(SG_DSR, 3); SGB(SG_MFMA, 1); SGB(SG_DSR, 3); SGB(SG_MFMA, 1); }
      }
    }
#pragma unroll
    for (int j = 0; j < NT; ++j) b[j] = nb[j];
    // stage 1: A_{d+2}, 3 + 3 + 2 DMAs; the barrier after the third row block
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      sa[i] = pick(sa8[i], 2 * PAR + 1);
      sb[i] = pick(sb8[i], 2 * PAR + 1);
    }
#pragma unroll
    for (int q = 0; q < NT - 1; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      const int nd = NT == 2 ? 4 : q < 2 ? 3 : 2, d0 = 3 * q;
#pragma unroll
      for (int k = 0; k < nd; ++k) dma(s_a2, 0, ka2, d0 + k);
      if (q & 1) a0 = frag(s_a, 1, wn + (q + 1) * 32 + lrow);
      else a1 = frag(s_a, 1, wn + (q + 1) * 32 + lrow);
      mfma_row((q & 1) ? a1 : a0, q);
      if (nd == 4) {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 2); SGB(SG_DSR, 2); SGB(SG_MFMA, 1); SGB(SG_VMEM, 2);
      } else if (nd == 3) {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1);
      } else {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
        SGB(SG_MFMA, 2);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    wait_vm<NDMA>();   // all but A_{d+2}'s: B_{d+1}, A_{d+1} and the scale loads are in
    wait_lgkm0();
    bare_barrier();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < NT; ++j) nb[j] = frag(s_b1, 0, wt + j * 32 + lrow);
    a0 = frag(s_a1, 0, wn + lrow);
    mfma_row(a1, NT - 1);
    SGB(SG_MFMA, 1); SGB(SG_DSR, 4); SGB(SG_MFMA, 1);
    if (NT == 4) { SGB(SG_DSR, 3); SGB(SG_MFMA, 1); SGB(SG_DSR, 3); SGB(SG_MFMA, 1); }
#pragma unroll
    for (int j = 0; j < NT; ++j) b[j] = nb[j];
    if (PAR == 1) {
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        sa8[i] = na8[i];
        sb8[i] = nb8[i];
      }
    }
    base = base + 2 >= Q_SLOTS ? base + 2 - Q_SLOTS : base + 2;
  };
  for (int d = 0; d < (HALF ? ns - 1 : ns); d += 2) {
    slice(d, std::integral_constant<int, 0>{});
    slice(d + 1, std::integral_constant<int, 1>{});
  }
  if constexpr (HALF) slice(ns - 1, std::integral_constant<int, 0>{});
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  store_tile<NT>(acc, smem, kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

template <int NT>
hipError_t launch_mx_ring(const uint8_t* xq, const uint8_t* xs, int T, int K, const uint8_t* w, const uint8_t* ws,
                          int N, uint16_t* kv, int tn0, int tiles_n, hipStream_t s, const GateEpi& ep) {
  const int tiles_t = (T + 64 * NT - 1) / (64 * NT);
  constexpr int lds = Q_LDS * NT / 4;
  const auto fn = K % 256 ? gemm_mx_ring_kernel<NT, true> : gemm_mx_ring_kernel<NT, false>;
  const hipError_t e = set_lds((const void*)fn, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(fn, dim3(tiles_n * tiles_t), dim3(THREADS), lds, s, xq, xs, T, K, w, ws, N, kv, tn0, tiles_n,
                     tiles_t, ep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_bf16(const void* x, int64_t T, int K, const void* w, int N, void* kv,
                            hipStream_t s, const GateEpi& ep) {
  const int tiles_n = (N + BM - 1) / BM;
  const int tiles_t = (int)((T + BN - 1) / BN);
  const dim3 grid(tiles_n * tiles_t), block(THREADS);
  hipError_t e;
  if (K % 64 == 0) {
    if ((e = set_lds((const void*)gemm_bf16_kernel<false>, Q_LDS)) != hipSuccess) return e;
    hipLaunchKernelGGL(gemm_bf16_kernel<false>, grid, block, Q_LDS, s, (const uint16_t*)x, (int)T, K,
                       (const uint16_t*)w, N, (uint16_t*)kv, tiles_n, tiles_t, ep);
  } else {
    if ((e = set_lds((const void*)gemm_bf16_kernel<true>, Q_LDS)) != hipSuccess) return e;
    hipLaunchKernelGGL(gemm_bf16_kernel<true>, grid, block, Q_LDS, s, (const uint16_t*)x, (int)T, K,
                       (const uint16_t*)w, N, (uint16_t*)kv, tiles_n, tiles_t, ep);
  }
  return hipGetLastError();
}

// Measured in us, 256x256 / 128x128 tiles: N 20480, K 2048: T 128 25.6 / 13.8, T
// 300 27 / 19, T 515 29.5 / 35.6, T 1000 57 / 48, T 8192 310 / 369; T 383, N 7808,
// K 384 12.0 / 5.2; T 6968, N 10112, K 640 76 / 68.
// The gate's epilogue has the 256x256 tile only.
hipError_t launch_gemm_mxfp8(const uint8_t* xq, const uint8_t* xs, int64_t T, int K, const uint8_t* w,
                             const uint8_t* ws, int N, void* kv, hipStream_t s, const GateEpi& ep) {
  uint16_t* out = (uint16_t*)kv;
  const int big = ep.hidden ? (N + 255) / 256 : big_columns(T, N, K, {8000, 1400, 3200, 950, 3200, 660});
  if (big) {
    const hipError_t e = launch_mx_ring<4>(xq, xs, (int)T, K, w, ws, N, out, 0, big, s, ep);
    if (e != hipSuccess || 256 * (int64_t)big >= N) return e;
  }
  return launch_mx_ring<2>(xq, xs, (int)T, K, w, ws, N, out, 2 * big, (N + 127) / 128 - 2 * big, s, ep);
}

}  // namespace engram
