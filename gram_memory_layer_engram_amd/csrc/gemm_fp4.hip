// Tiled projection GEMMs with MXFP4 weights: kv[T, N] = bf16(x . deq(W)^T), x
// bf16 (gemm_fp4_bf16_kernel) or MXFP8 (gemm_fp4_mx_kernel), K % 128 == 0.
//
// The block (256 W rows x 256 tokens, four waves of 128x128 on 32x32 MFMA
// tiles), tile order, DMAs and epilogue are the other tiled GEMMs' (gemm.hip).
// W stays e2m1 all the way into LDS: a 128-byte LDS row of W holds 256 k, so a
// 32 KiB chunk of W serves four bf16 slices of x (64 k) or two MXFP8 slices
// (128 k), and a slice moves 40 (48) KiB from L2 instead of 64, which is what
// bounds those kernels. LDS: two slots for W chunks, a ring of three or
// four for x.
// Where K % 256 == 128 the last chunk is half: its rows' second 64 bytes are
// the next row's (zeros past the tile), as the second half of its scale bytes
// is, and the loop ends before the slices that would use them.
//
//  * bf16 x: lane (row l%32, half h = l/32) reads, per slice, the 16 bytes of k
//    32h .. 32h+31 of its row: one scale group. v_cvt_scalef32_pk_bf16_fp4 turns
//    its word kk into the A fragment of v_mfma_f32_32x32x16_bf16 number kk (k
//    32h+8kk .. +7; the order of k inside a product is free as long as x follows
//    it: its fragment kk is piece 4h+kk). The 16 conversions of a row block run
//    under the MFMAs, one sub-step ahead.
//  * MXFP8 x: v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes as they are:
//    lane group g holds k 32g .. 32g+31 of the fp4 operand in its 16 bytes, of
//    the fp8 operand k 16g.. and 32+16g.., and its E8M0 bytes scale k block
//    [32g, 32g+32) of its own row.
//
// Measured at N 20480, K 2048, T 8192: bf16 x 485-527 us (1.30-1.42 PFLOP/s;
// matrix cores busy 68% of the cycles, at the 1.9 GHz that the chip sustains
// with them busy), against 517 us for the weight expanded to bf16 and
// multiplied by the bf16 kernel; MXFP8 x 282-302 us (2.3-2.4 PFLOP/s).
#include <type_traits>

#include "gemm_tile.h"

namespace engram {

namespace {

constexpr int kWSlots = 2;
// A block is 64 * NT W rows x 64 * NT tokens: 256 x 256, or 128 x 128 with two
// workgroups on a compute unit (launch_gemm_mxfp4). x is fetched LA slices
// ahead, into a ring of LA + 1: two fill LDS; three where there is one 128 x
// 128 workgroup for a compute unit and no other to cover a late slice (N 20480,
// T 128, bf16 / MXFP8 x: K 2048 18.6 -> 15.5 / 11.5 -> 10.5 us, K 4096 33.4 ->
// 26.9 / 20.6 -> 20.1; four, or a third slot for W, gave no more).
constexpr int fp4_lds(int nt, int la) { return (kWSlots + la + 1) * 64 * nt * Q_ROW; }
static_assert(fp4_lds(4, 2) == Q_LDS && 2 * fp4_lds(2, 2) <= Q_LDS, "LDS budget");
constexpr int SG_VALU = 0x002;

template <int V> using Int = std::integral_constant<int, V>;

template <int NT, bool HALF, int LA>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(NT == 4 ? 1 : 2, NT == 4 ? 1 : 2)))
void gemm_fp4_bf16_kernel(const uint16_t* __restrict__ x, int T, int K, const uint8_t* __restrict__ w,
                          const uint8_t* __restrict__ ws, int N, uint16_t* __restrict__ kv, int tn0, int tiles_n,
                          int tiles_t, GateEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int tn, tt;
  tile_of(blockIdx.x, tiles_n, tiles_t, tn, tt);
  constexpr int TILE = 64 * NT, CH = TILE * Q_ROW, NDMA = 2 * NT;   // a chunk or slice in LDS, a wave's DMAs for it
  constexpr int XBASE = kWSlots * CH;
  const int n0 = (tn0 + tn) * TILE, t0 = tt * TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * (32 * NT), wt = (wave & 1) * (32 * NT);
  const uint32_t wpitch = (uint32_t)K / 2u, xpitch = (uint32_t)K * 2u, kb = (uint32_t)K / 32u;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * wpitch, (uint32_t)min(TILE, N - n0) * wpitch);
  const rsrc_t rb = make_rsrc(x + (int64_t)t0 * K, (uint32_t)min(TILE, T - t0) * xpitch);
  const rsrc_t rs = make_rsrc(ws + (int64_t)n0 * kb, (uint32_t)min(TILE, N - n0) * kb);
  const uint32_t ooba = (uint32_t)TILE * wpitch, oobb = (uint32_t)TILE * xpitch;   // at or past the ranges
  const int nk = K / 64, nc = K / 256 + HALF;   // x slices (even), W chunks

  const dma::Lane la = dma::lane_of(wave, lane, wpitch), lb = dma::lane_of(wave, lane, xpitch);
  auto dma_w = [&](int slot, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(smem + slot + (wave + 4 * i) * 1024), 16,
                                             dma::voffset(la, i, kofs, wpitch, ooba, false), 0, 0, 0);
  };
  auto dma_x = [&](int slot, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(smem + slot + (wave + 4 * i) * 1024), 16,
                                             dma::voffset(lb, i, kofs, xpitch, oobb, false), 0, 0, 0);
  };

  const int lrow = lane & 31, lhalf = lane >> 5;
  const int fsw = (lrow >> 1) & 7;
  // the 8 scale bytes of a chunk (256 k) of this lane's four rows; byte
  // 2*PAR + h is slice PAR's
  uint32_t srow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) srow[i] = (uint32_t)(wn + i * 32 + lrow) * kb;
  auto scales8 = [&](int c, u32x2 (&s8)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) s8[i] = __builtin_amdgcn_raw_buffer_load_b64(rs, srow[i] + 8u * (uint32_t)c, 0, 0);
  };
  // byte 2*par + h in the exponent field of an fp32 (the conversion reads no
  // other bits of its scale)
  const uint32_t lsh = 8u * (uint32_t)lhalf;
  auto pick = [&](const u32x2& v, int par) {
    return __uint_as_float(((par < 2 ? v.x : v.y) >> ((uint32_t)(16 * (par & 1)) + lsh)) << 23);
  };

  f32x16 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  bf16x8_t a[2][NT], b[2][NT];
  i32x4 raw[NT];
  float sc[NT];
  auto read_raw = [&](int slot, int par, int i) {
    raw[i] = *reinterpret_cast<const i32x4*>(smem + slot + (wn + i * 32 + lrow) * Q_ROW +
                                             (((2 * par + lhalf) ^ fsw) << 4));
  };
  auto read_x = [&](int slot, int kk, int c, int j) {
    b[c][j] = *reinterpret_cast<const bf16x8_t*>(smem + slot + (wt + j * 32 + lrow) * Q_ROW +
                                                 (((4 * lhalf + kk) ^ fsw) << 4));
  };
  auto convert = [&](int kk, int c, int i) {
    const uint32_t v = (uint32_t)raw[i][kk];
    const i32x4 f = {(int)fp4_pair_to_bf16<0>(v, sc[i]), (int)fp4_pair_to_bf16<1>(v, sc[i]),
                     (int)fp4_pair_to_bf16<2>(v, sc[i]), (int)fp4_pair_to_bf16<3>(v, sc[i])};
    a[c][i] = __builtin_bit_cast(bf16x8_t, f);
  };
  auto mfma_row = [&](int c, int i) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(a[c][i], b[c][j], acc[i][j], 0, 0, 0);
  };
  auto wslot = [](int c) { return (c & 1) * CH; };

  // prologue: W chunk 0, x slices 0 .. LA - 1; W and x slice 0 waited for
  u32x2 s8[NT], n8[NT];
  scales8(0, s8);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma_w(0, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma_x(XBASE, 0u, i);
#pragma unroll
  for (int m = 1; m < LA; ++m)
#pragma unroll
    for (int i = 0; i < NDMA; ++i) dma_x(XBASE + m * CH, m < 2 || m < nk ? (uint32_t)(m * Q_ROW) : oobb, i);
  wait_vm<(LA - 1) * NDMA>();
  // a use here keeps the scale loads ahead of the DMAs
#pragma unroll
  for (int i = 0; i < NT; ++i) asm volatile("" : "+v"(s8[i]));
  bare_barrier();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    read_raw(0, 0, i);
    sc[i] = pick(s8[i], 0);
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) read_x(XBASE, 0, 0, j);
#pragma unroll
  for (int i = 0; i < NT; ++i) convert(0, 0, i);

  int xb = 0;   // d % (LA + 1)
  // slice d (64 k), par = d % 4: x of slice d+LA and, in the chunk's first
  // three slices, W of the next chunk are fetched; the barrier that publishes
  // slice d+1 sits after the first 4 of the last 16 MFMAs.
  auto slice = [&](int d, auto par) {
    constexpr int PAR = decltype(par)::value;
    const int c = d >> 2;
    auto xslot = [&](int m) { const int v = xb + m; return XBASE + (v > LA ? v - LA - 1 : v) * CH; };
    const int sb = xslot(0), sb1 = xslot(1), sb2 = xslot(LA);
    const uint32_t kx = d + LA < nk ? (uint32_t)(d + LA) * Q_ROW : oobb;
    const uint32_t kw = c + 1 < nc ? (uint32_t)(c + 1) * Q_ROW : ooba;
    if (PAR == 0) scales8(min(c + 1, nc - 1), n8);   // the last chunk reloads itself, unused
    // sub-steps 0..2: MFMAs of sub-step kk, fragments of kk+1
#pragma unroll
    for (int kk = 0; kk < 3; ++kk) {
#pragma unroll
      for (int q = 0; q < NT; ++q) {
        __builtin_amdgcn_sched_barrier(0);
        // W: 3 + 3 + 2 (2 + 1 + 1) DMAs over a chunk's first three slices
        constexpr int w0 = NT == 4 ? 3 * PAR : PAR + (PAR > 0), wd = NT == 4 ? (PAR == 2 ? 2 : 3) : (PAR ? 1 : 2);
        const bool dw = PAR < 3 && kk == 0 && q < wd;
        if (dw) dma_w(wslot(c + 1), kw, w0 + q);
        const int x0 = kk * NT + q - (NT == 4);   // x: one each from (kk 0, q 1 or 0) on
        const bool dx = x0 >= 0 && x0 < NDMA;
        if (dx) dma_x(sb2, kx, x0);
        read_x(sb, kk + 1, (kk + 1) & 1, q);
        convert(kk + 1, (kk + 1) & 1, q);
        mfma_row(kk & 1, q);
        SGB(SG_MFMA, 1);
        if (dw) SGB(SG_VMEM, 1);
        if (dx) SGB(SG_VMEM, 1);
        if (NT == 4) { SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VALU, 4); SGB(SG_MFMA, 1); }
        else { SGB(SG_DSR, 1); SGB(SG_VALU, 4); SGB(SG_MFMA, 1); }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    mfma_row(1, 0);
    __builtin_amdgcn_sched_barrier(0);
    // only the last LA - 1 slices' x DMAs may still fly; the next chunk's last W
    // DMA went out beside the first of slice d-1's, in whichever order
    wait_vm<(LA - 1) * NDMA - (LA > 2 && PAR == 3)>();
    wait_lgkm0();
    bare_barrier();
    // the rest of sub-step 3: slice d+1's W words, first x fragments, conversions
    const int sw1 = wslot(PAR == 3 ? c + 1 : c);
    auto next_w = [&]() {
#pragma unroll
      for (int i = 0; i < NT; ++i) read_raw(sw1, (PAR + 1) & 3, i);
    };
    auto next_x = [&]() {
#pragma unroll
      for (int j = 0; j < NT; ++j) read_x(sb1, 0, 0, j);
#pragma unroll
      for (int i = 0; i < NT; ++i) sc[i] = PAR == 3 ? pick(n8[i], 0) : pick(s8[i], (PAR + 1) & 3);
    };
    __builtin_amdgcn_sched_barrier(0);
    next_w();
    if constexpr (NT == 4) {
      mfma_row(1, 1);
      SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 2);
      __builtin_amdgcn_sched_barrier(0);
      next_x();
      mfma_row(1, 2);
      SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 2);
      __builtin_amdgcn_sched_barrier(0);
    } else {
      next_x();
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) convert(0, 0, i);
    mfma_row(1, NT - 1);
    if (NT == 4) {
      SGB(SG_MFMA, 1); SGB(SG_VALU, 5); SGB(SG_MFMA, 1); SGB(SG_VALU, 5); SGB(SG_MFMA, 1); SGB(SG_VALU, 5);
      SGB(SG_MFMA, 1);
    }
    if (PAR == 3) {
#pragma unroll
      for (int i = 0; i < NT; ++i) s8[i] = n8[i];
    }
    xb = xb + 1 > LA ? 0 : xb + 1;
  };
  for (int d = 0; d < (HALF ? nk - 2 : nk); d += 4) {
    slice(d, Int<0>{});
    slice(d + 1, Int<1>{});
    slice(d + 2, Int<2>{});
    slice(d + 3, Int<3>{});
  }
  if constexpr (HALF) {
    slice(nk - 2, Int<0>{});
    slice(nk - 1, Int<1>{});
  }
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  store_tile<NT>(acc, smem, kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

template <int NT, bool HALF, int LA>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(NT == 4 ? 1 : 2, NT == 4 ? 1 : 2)))
void gemm_fp4_mx_kernel(const uint8_t* __restrict__ xq, const uint8_t* __restrict__ xs, int T, int K,
                        const uint8_t* __restrict__ w, const uint8_t* __restrict__ ws, int N,
                        uint16_t* __restrict__ kv, int tn0, int tiles_n, int tiles_t, GateEpi ep) {
  extern __shared__ __attribute__((aligned(1024))) char smem[];
  int tn, tt;
  tile_of(blockIdx.x, tiles_n, tiles_t, tn, tt);
  constexpr int TILE = 64 * NT, CH = TILE * Q_ROW, NDMA = 2 * NT;   // a chunk or slice in LDS, a wave's DMAs for it
  constexpr int XBASE = kWSlots * CH;
  const int n0 = (tn0 + tn) * TILE, t0 = tt * TILE;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = (wave >> 1) * (32 * NT), wt = (wave & 1) * (32 * NT);
  const uint32_t wpitch = (uint32_t)K / 2u, xpitch = (uint32_t)K, kb = (uint32_t)K / 32u;
  const rsrc_t ra = make_rsrc(w + (int64_t)n0 * wpitch, (uint32_t)min(TILE, N - n0) * wpitch);
  const rsrc_t rb = make_rsrc(xq + (int64_t)t0 * xpitch, (uint32_t)min(TILE, T - t0) * xpitch);
  const rsrc_t rsa = make_rsrc(ws + (int64_t)n0 * kb, (uint32_t)min(TILE, N - n0) * kb);
  const rsrc_t rsb = make_rsrc(xs + (int64_t)t0 * kb, (uint32_t)min(TILE, T - t0) * kb);
  const uint32_t ooba = (uint32_t)TILE * wpitch, oobb = (uint32_t)TILE * xpitch;
  const int ns = K / 128, nc = K / 256 + HALF;   // x slices, W chunks

  const dma::Lane la = dma::lane_of(wave, lane, wpitch), lb = dma::lane_of(wave, lane, xpitch);
  auto dma_w = [&](int slot, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(smem + slot + (wave + 4 * i) * 1024), 16,
                                             dma::voffset(la, i, kofs, wpitch, ooba, false), 0, 0, 0);
  };
  auto dma_x = [&](int slot, uint32_t kofs, int i) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr_t)(smem + slot + (wave + 4 * i) * 1024), 16,
                                             dma::voffset(lb, i, kofs, xpitch, oobb, false), 0, 0, 0);
  };

  const int lrow = lane & 31, lg = lane >> 5;
  const int fsw = (lrow >> 1) & 7;
  // the 8 scale bytes of a chunk (four stages of 64 k) of this lane's W and
  // token rows; lane group g takes byte 2*stage + g
  uint32_t arow[NT], brow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) arow[i] = (uint32_t)(wn + i * 32 + lrow) * kb;
#pragma unroll
  for (int j = 0; j < NT; ++j) brow[j] = (uint32_t)(wt + j * 32 + lrow) * kb;
  auto scales8 = [&](int c, u32x2 (&a8)[NT], u32x2 (&b8)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a8[i] = __builtin_amdgcn_raw_buffer_load_b64(rsa, arow[i] + 8u * (uint32_t)c, 0, 0);
      b8[i] = __builtin_amdgcn_raw_buffer_load_b64(rsb, brow[i] + 8u * (uint32_t)c, 0, 0);
    }
  };
  const uint32_t lsh = (uint32_t)lg * 8u;
  auto pick = [&](const u32x2& v, int u) {   // u static: byte 2u + lg
    return (int)(((u < 2 ? v.x : v.y) >> ((uint32_t)(16 * (u & 1)) + lsh)) & 0xffu);
  };
  // W fragment of stage u (0..3) of a chunk, x fragment of half h of a slice
  auto wfrag = [&](int slot, int u, int i) {
    return *reinterpret_cast<const i32x4*>(smem + slot + (wn + i * 32 + lrow) * Q_ROW + (((2 * u + lg) ^ fsw) << 4));
  };
  auto xfrag = [&](int slot, int h, int j) {
    const char* base = smem + slot + (wt + j * 32 + lrow) * Q_ROW;
    const i32x4 lo = *reinterpret_cast<const i32x4*>(base + (((4 * h + lg) ^ fsw) << 4));
    const i32x4 hi = *reinterpret_cast<const i32x4*>(base + (((4 * h + 2 + lg) ^ fsw) << 4));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  f32x16 acc[NT][NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  i32x4 a[NT], na[NT];
  i32x8 b[NT], nb[NT];
  int sa[NT], sb[NT];
  auto mfma_row = [&](int i) {
    const i32x8 wa = __builtin_shufflevector(a[i], a[i], 0, 1, 2, 3, 0, 1, 2, 3);   // fp4: the first four words
#pragma unroll
    for (int j = 0; j < NT; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wa, b[j], acc[i][j], 4, 0, 0, sa[i], 0, sb[j]);
  };
  auto wslot = [](int c) { return (c & 1) * CH; };

  u32x2 sa8[NT], sb8[NT], na8[NT], nb8[NT];
  scales8(0, sa8, sb8);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma_w(0, 0u, i);
#pragma unroll
  for (int i = 0; i < NDMA; ++i) dma_x(XBASE, 0u, i);
#pragma unroll
  for (int m = 1; m < LA; ++m)
#pragma unroll
    for (int i = 0; i < NDMA; ++i) dma_x(XBASE + m * CH, m < 2 || m < ns ? (uint32_t)(m * Q_ROW) : oobb, i);
  wait_vm<(LA - 1) * NDMA>();
#pragma unroll
  for (int i = 0; i < NT; ++i) asm volatile("" : "+v"(sa8[i]));
#pragma unroll
  for (int j = 0; j < NT; ++j) asm volatile("" : "+v"(sb8[j]));
  bare_barrier();
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    a[i] = wfrag(0, 0, i);
    sa[i] = pick(sa8[i], 0);
    b[i] = xfrag(XBASE, 0, i);
    sb[i] = pick(sb8[i], 0);
  }

  int xb = 0;   // d % (LA + 1)
  // slice d (two stages of 64 k), par = d % 2: x of slice d+LA goes out in the
  // last six quarters, W of the next chunk in the first four of an even slice
  auto slice = [&](int d, auto par) {
    constexpr int PAR = decltype(par)::value;
    const int c = d >> 1;
    auto xslot = [&](int m) { const int v = xb + m; return XBASE + (v > LA ? v - LA - 1 : v) * CH; };
    const int s_x = xslot(0), s_x1 = xslot(1), s_x2 = xslot(LA);
    const uint32_t kx = d + LA < ns ? (uint32_t)(d + LA) * Q_ROW : oobb;
    const uint32_t kw = c + 1 < nc ? (uint32_t)(c + 1) * Q_ROW : ooba;
    if (PAR == 0) scales8(min(c + 1, nc - 1), na8, nb8);   // the last chunk reloads itself, unused
    // stage 0; stage 1's fragments are read ahead
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      if (PAR == 0) {
        dma_w(wslot(c + 1), kw, 2 * q);
        dma_w(wslot(c + 1), kw, 2 * q + 1);
      } else {
#pragma unroll
        for (int k = 0; k < NDMA / NT; ++k) dma_x(s_x2, kx, NDMA / NT * q + k);
      }
      na[q] = wfrag(wslot(c), 2 * PAR + 1, q);
      nb[q] = xfrag(s_x, 1, q);
      mfma_row(q);
      if (NT == 4) {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_DSR, 1);
        SGB(SG_MFMA, 1); SGB(SG_DSR, 1); SGB(SG_MFMA, 1);
      } else {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 2); SGB(SG_DSR, 3); SGB(SG_MFMA, 1);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a[i] = na[i];
      sa[i] = pick(sa8[i], 2 * PAR + 1);
      b[i] = nb[i];
      sb[i] = pick(sb8[i], 2 * PAR + 1);
    }
    // stage 1; the barrier that publishes slice d+1 after half its row blocks
#pragma unroll
    for (int q = 0; q < NT / 2; ++q) {
      __builtin_amdgcn_sched_barrier(0);
      if (PAR == 0) {
#pragma unroll
        for (int k = 0; k < 2 * NDMA / NT; ++k) dma_x(s_x2, kx, 2 * NDMA / NT * q + k);
      }
      mfma_row(q);
      if (PAR == 0) {
        SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1);
        if (NT == 4) { SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); SGB(SG_MFMA, 1); SGB(SG_VMEM, 1); }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    // in flight may be x of slices d+2 .. d+LA and, in an even slice, the W
    // chunk after this slice's (not needed before the next slice's end)
    if (PAR == 0) wait_vm<LA * NDMA>();
    else wait_vm<(LA - 1) * NDMA>();
    wait_lgkm0();
    bare_barrier();
    const int sw1 = wslot(PAR == 1 ? c + 1 : c);
    constexpr int u1 = PAR == 1 ? 0 : 2;
#pragma unroll
    for (int q = NT / 2; q < NT; ++q) {
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 2 * q - NT; i < 2 * q - NT + 2; ++i) {
        na[i] = wfrag(sw1, u1, i);
        nb[i] = xfrag(s_x1, 0, i);
      }
      mfma_row(q);
      if (NT == 4) {
        SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 1); SGB(SG_DSR, 2); SGB(SG_MFMA, 1); SGB(SG_DSR, 2);
        SGB(SG_MFMA, 1);
      } else {
        SGB(SG_MFMA, 1); SGB(SG_DSR, 6); SGB(SG_MFMA, 1);
      }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      a[i] = na[i];
      if (PAR == 1) sa8[i] = na8[i];
      sa[i] = pick(sa8[i], u1);
      b[i] = nb[i];
      if (PAR == 1) sb8[i] = nb8[i];
      sb[i] = pick(sb8[i], u1);
    }
    xb = xb + 1 > LA ? 0 : xb + 1;
  };
  for (int d = 0; d < (HALF ? ns - 1 : ns); d += 2) {
    slice(d, Int<0>{});
    slice(d + 1, Int<1>{});
  }
  if constexpr (HALF) slice(ns - 1, Int<0>{});
  __builtin_amdgcn_sched_barrier(0);
  wait_vm<0>();   // the zero-fill DMAs of the last slices land before LDS is reused
  store_tile<NT>(acc, smem, kv, T, N, t0, n0, wn, wt, lane, wave, ep);
}

template <int NT, bool HALF, int LA>
hipError_t launch_half(const void* x, const uint8_t* xs, int T, int K, const uint8_t* w, const uint8_t* ws, int N,
                       uint16_t* kv, int tn0, int tiles_n, hipStream_t s, const GateEpi& ep) {
  const int tiles_t = (T + 64 * NT - 1) / (64 * NT);
  const dim3 grid(tiles_n * tiles_t), block(THREADS);
  constexpr int lds = fp4_lds(NT, LA);
  hipError_t e;
  if (xs) {
    const auto fn = gemm_fp4_mx_kernel<NT, HALF, LA>;
    if ((e = set_lds((const void*)fn, lds)) != hipSuccess) return e;
    hipLaunchKernelGGL(fn, grid, block, lds, s, (const uint8_t*)x, xs, T, K, w, ws, N, kv, tn0, tiles_n, tiles_t, ep);
  } else {
    const auto fn = gemm_fp4_bf16_kernel<NT, HALF, LA>;
    if ((e = set_lds((const void*)fn, lds)) != hipSuccess) return e;
    hipLaunchKernelGGL(fn, grid, block, lds, s, (const uint16_t*)x, T, K, w, ws, N, kv, tn0, tiles_n, tiles_t, ep);
  }
  return hipGetLastError();
}

// The half chunk at the end is code of its own behind the loop: one that the
// loop leaves early for cost the accumulators' registers (1000 spilled).
template <int NT, int LA>
hipError_t launch_tile(const void* x, const uint8_t* xs, int T, int K, const uint8_t* w, const uint8_t* ws, int N,
                       uint16_t* kv, int tn0, int tiles_n, hipStream_t s, const GateEpi& ep) {
  return K % 256 ? launch_half<NT, true, LA>(x, xs, T, K, w, ws, N, kv, tn0, tiles_n, s, ep)
                 : launch_half<NT, false, LA>(x, xs, T, K, w, ws, N, kv, tn0, tiles_n, s, ep);
}

}  // namespace

// Measured in us, 256x256 / 128x128 tiles: bf16 x, N 20480, K 2048: T 128 40 /
// 15.5, T 515 47 / 53, T 1000 91 / 73, T 8192 500 / 550; T 6164, N 10656, K 512 89
// / 76; MXFP8 x: T 128 25 / 10.5, T 515 29 / 32, T 8192 300 / 327, K 512 67 / 52.
// 256x128 tiles came within 2% of the better of the two at best, and went.
static int fp4_big_columns(int64_t T, int N, int K, bool x_mxfp8) {
  return big_columns(T, N, K, x_mxfp8 ? TileTimes{8000, 1370, 3100, 830, 1500, 570}
                                      : TileTimes{7000, 2700, 3000, 1540, 3400, 750});
}

bool gemm_mxfp4_big_tiles(int64_t T, int N, int K) { return fp4_big_columns(T, N, K, false) == (N + 255) / 256; }

// The gate's epilogue has the 256x256 tile only.
hipError_t launch_gemm_mxfp4(const void* x, const uint8_t* xs, int64_t T, int K, const uint8_t* w,
                             const uint8_t* ws, int N, void* kv, hipStream_t s, const GateEpi& ep) {
  const int big = ep.hidden ? (N + 255) / 256 : fp4_big_columns(T, N, K, xs != nullptr);
  if (big) {
    const hipError_t e = launch_tile<4, 2>(x, xs, (int)T, K, w, ws, N, (uint16_t*)kv, 0, big, s, ep);
    if (e != hipSuccess || 256 * (int64_t)big >= N) return e;
  }
  const int tn0 = 2 * big, tiles_n = (N + 127) / 128 - tn0;
  return tiles_n * ((T + 127) / 128) <= dev_info().num_cus
             ? launch_tile<2, 3>(x, xs, (int)T, K, w, ws, N, (uint16_t*)kv, tn0, tiles_n, s, ep)
             : launch_tile<2, 2>(x, xs, (int)T, K, w, ws, N, (uint16_t*)kv, tn0, tiles_n, s, ep);
}

}  // namespace engram
