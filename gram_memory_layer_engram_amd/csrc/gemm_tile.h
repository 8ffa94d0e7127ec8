// What the tiled projection GEMMs share (gemm.hip: bf16 and MXFP8 weights,
// gemm_fp4.hip: MXFP4 weights): block geometry, tile order, waits and the
// epilogue. The design is described in gemm.hip.
#pragma once

#include "common.h"
#include "gemm_dma.h"

namespace engram {

namespace {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

constexpr int BM = 256;      // W rows per block
constexpr int BN = 256;      // tokens per block
constexpr int THREADS = 256;
constexpr int LDS_BYTES = 128 * 1024;            // the epilogue's staging tile (rings: Q_LDS)
static_assert(BN * 512 == LDS_BYTES, "epilogue staging tile");
// rings: 64-element bf16 (128-element MXFP8) k slices (128-byte LDS rows of 8 pieces, piece p of row
// r at p ^ ((r >> 1) & 7)); each operand's slice is a 32 KiB chunk in a ring
// of five
constexpr int Q_ROW = 128;
constexpr int Q_CHUNK = BM * Q_ROW;
constexpr int Q_SLOTS = 5;
constexpr int Q_LDS = Q_SLOTS * Q_CHUNK;         // 160 KiB
constexpr int Q_DMA = Q_CHUNK / (THREADS * 16);  // DMA instructions per wave per chunk
static_assert(Q_DMA == 8 && Q_LDS >= LDS_BYTES, "bf16 ring");
constexpr int GROUP_T = 4;
constexpr uint32_t RSRC_FLAGS = 0x00020000u;

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes, RSRC_FLAGS);
}

__device__ __forceinline__ void tile_of(int bid, int tiles_n, int tiles_t, int& tn, int& tt) {
  const int total = tiles_n * tiles_t;
  const int q = total / 8, r = total % 8;
  const int xcd = bid % 8, slot = bid / 8;
  const int logical = (xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q) + slot;
  const int per_group = GROUP_T * tiles_n;
  const int group = logical / per_group;
  const int first_t = group * GROUP_T;
  const int gsize = min(tiles_t - first_t, GROUP_T);
  const int in_group = logical - group * per_group;
  tt = first_t + in_group % gsize;
  tn = in_group / gsize;
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void wait_lgkm0() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }
// A bare workgroup barrier: unlike __syncthreads() it does not first wait
// for every outstanding vector load, so later stages keep streaming.
__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" ::: "memory"); }

#define SGB(mask, n) __builtin_amdgcn_sched_group_barrier(mask, n, 0)
constexpr int SG_MFMA = 0x008, SG_VMEM = 0x010, SG_DSR = 0x100;

// 16 bytes of the output tile, stored non-temporal: the kernel never reads
// kv back, and streaming it past the L2 keeps the operand lines there (the
// long-prefill MXFP8 GEMM, 2.2 GiB of kv: 3.15 -> 2.98 ms; the prefill
// shapes unchanged).
__device__ __forceinline__ void store_nt(uint16_t* dst, const uint4& v) {
  typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
  const u32x4_t w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(dst));
}

// Write the block's accumulators: converted with v_cvt_pk_bf16_f32 (one
// instruction per pair instead of a dozen for the bit-level rounding: 644 ->
// 614 us for the prefill GEMM), staged in LDS as [token][n]
// (512-byte rows; 16-byte chunk c of row t at c ^ (t & 31)), then go over
// whole rows. The caller has drained its DMAs; LDS is free after the first
// barrier here. Rows past T are not written.
//  * plain (ep.hidden == nullptr): store the rows into kv [T, N] (N % 4 == 0,
//    so a row's last chunk may be half);
//  * gate epilogue (dim % 256 == 0, so a tile lies inside one key block or
//    the value block): value tiles go to ep.value [T, dim]; key tiles are
//    not stored but reduced, per token, to the gate's two kv-side sums over
//    the tile's 256 columns, sum hidden*q*k*key and sum key^2 of the
//    bf16-rounded keys ("vllm.models.deepseek_v41.amd.engram",
//    _engram_gate_partials_kernel, at tile granularity), into
//    ep.part[(h*T + t) * (dim/256) + tile].
// NT: 32-row and 32-token blocks of a wave (4: the 256x256 tile; 2: 128x128,
// the plain store only).
template <int NT = 4>
__device__ __forceinline__ void store_tile(f32x16 (&acc)[NT][NT], char* smem, uint16_t* __restrict__ kv,
                                           int T, int N, int t0, int n0, int wn, int wt, int lane,
                                           int wave, const GateEpi& ep) {
  constexpr int RB = 128 * NT, CPR = 8 * NT;   // bytes and 16-byte chunks of a staged row
  const int lrow = lane & 31, lhalf = lane >> 5;
  wait_lgkm0();
  bare_barrier();
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int t = wt + j * 32 + lrow;
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        // accumulator r of lane l: n = 8*(r/4) + 4*(l/32) + r%4, token = l%32
        const int n = wn + i * 32 + 8 * g + 4 * lhalf;
        uint2 o;
        o.x = cvt_pk_bf16(acc[i][j][4 * g + 0], acc[i][j][4 * g + 1]);
        o.y = cvt_pk_bf16(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3]);
        *reinterpret_cast<uint2*>(smem + t * RB + (((n >> 3) ^ (t & (CPR - 1))) << 4) + (n & 7) * 2) = o;
      }
  }
  wait_lgkm0();
  bare_barrier();
  const int c = lane & (CPR - 1);
  auto lds_row = [&](int t) {
    return *reinterpret_cast<const uint4*>(smem + t * RB + ((c ^ (t & (CPR - 1))) << 4));
  };
  if (NT < 4 || !ep.hidden) {
    const int n = n0 + c * 8;
#pragma unroll 4
    for (int it = 0; it < 2 * NT * NT; ++it) {
      const int t = wave * (16 * NT) + it * (64 / CPR) + lane / CPR;
      const uint4 v = lds_row(t);
      if (t0 + t < T) {
        uint16_t* dst = kv + (int64_t)(t0 + t) * N + n;
        if (n + 8 <= N) store_nt(dst, v);
        else if (n + 4 <= N) *reinterpret_cast<uint2*>(dst) = make_uint2(v.x, v.y);
      }
    }
    return;
  }
  const int key_cols = ep.hc * ep.dim;
  if (n0 >= key_cols) {
    // value tile
    const int d = n0 - key_cols + c * 8;
#pragma unroll 4
    for (int it = 0; it < 32; ++it) {
      const int t = wave * 64 + it * 2 + (lane >> 5);
      const uint4 v = lds_row(t);
      if (t0 + t < T) store_nt(ep.value + (int64_t)(t0 + t) * ep.dim + d, v);
    }
    return;
  }
  // key tile of copy h, columns d0 .. d0+255 of that copy. Lane group g =
  // lane/16 of wave w takes rows t = 64w + 4r + g (r = 0..15: the four
  // groups read consecutive rows, which the LDS swizzle keeps on distinct
  // banks); lane c16 = lane%16 takes the 16-byte pieces c16 and 16 + c16 of
  // each row (columns 8*c16.. and 128 + 8*c16..), so a load instruction
  // covers 256 contiguous bytes of four rows.
  const int h = n0 / ep.dim, d0 = n0 - h * ep.dim;
  const int g = lane >> 4, c16 = lane & 15;
  float qk[16];
  {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int d = d0 + half * 128 + c16 * 8;
      const uint4 q8 = *reinterpret_cast<const uint4*>(ep.q + h * ep.dim + d);
      const uint4 k8 = *reinterpret_cast<const uint4*>(ep.k + h * ep.dim + d);
      const uint32_t qw[4] = {q8.x, q8.y, q8.z, q8.w}, kw[4] = {k8.x, k8.y, k8.z, k8.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        qk[half * 8 + 2 * e] = bf16lo(qw[e]) * bf16lo(kw[e]);
        qk[half * 8 + 2 * e + 1] = bf16hi(qw[e]) * bf16hi(kw[e]);
      }
    }
  }
  const int tiles = ep.dim / 256, tile = d0 / 256;
  // all 32 hidden pieces of this thread in flight at once (the accumulators
  // are dead, their registers free), then the reductions
  uint4 hid[16][2];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int t = wave * 64 + 4 * r + g;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      hid[r][half] = make_uint4(0, 0, 0, 0);
      if (t0 + t < T)
        hid[r][half] = *reinterpret_cast<const uint4*>(ep.hidden + ((int64_t)(t0 + t) * ep.hc + h) * ep.dim + d0 +
                                                       half * 128 + c16 * 8);
    }
  }
  // per-lane sums of this lane's 16 columns, one pair per row r
  float dts[16], kss[16];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int t = wave * 64 + 4 * r + g;
    float dt = 0.f, ks = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int ch = half * 16 + c16;
      const uint4 kv8 = *reinterpret_cast<const uint4*>(smem + t * 512 + ((ch ^ (t & 31)) << 4));
      const uint4 h8 = hid[r][half];
      const uint32_t kw[4] = {kv8.x, kv8.y, kv8.z, kv8.w}, hw[4] = {h8.x, h8.y, h8.z, h8.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float k0 = bf16lo(kw[e]), k1 = bf16hi(kw[e]);
        ks = fmaf(k0, k0, ks);
        ks = fmaf(k1, k1, ks);
        dt = fmaf(bf16lo(hw[e]) * qk[half * 8 + 2 * e], k0, dt);
        dt = fmaf(bf16hi(hw[e]) * qk[half * 8 + 2 * e + 1], k1, dt);
      }
    }
    dts[r] = dt;
    kss[r] = ks;
  }
  // Sum over the 16 lanes of each group for all 16 rows at once: at each
  // step lane c16 keeps the half of its rows selected by bit w of c16 and
  // adds the partner's (lane c16^w) copy of them, so 15 exchanges per sum;
  // lane c16 ends with row r = c16, in a fixed order. (With 32 lanes per row
  // the exchanges double, 62 shuffles against 30: 633 -> 625 us at the
  // prefill shape; 8 lanes per row, 14 shuffles but 128-byte row pieces per
  // load, measured 642 us.)
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
    const bool upper = (c16 & w) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float rd = __shfl_xor(upper ? dts[i] : dts[i + w], w, 64);
      const float rk = __shfl_xor(upper ? kss[i] : kss[i + w], w, 64);
      dts[i] = (upper ? dts[i + w] : dts[i]) + rd;
      kss[i] = (upper ? kss[i + w] : kss[i]) + rk;
    }
  }
  const int t = wave * 64 + 4 * c16 + g;
  if (t0 + t < T) ep.part[((int64_t)h * T + t0 + t) * tiles + tile] = make_float2(dts[0], kss[0]);
}

// How many columns of 256 W rows are stored by 256x256 tiles, the rest by
// 128x128 ones (a second launch): by the rounds that each needs and a round's
// time, an offset (launch, first DMAs, epilogue) and so much a 128-k slice. All,
// none, or as many as fill whole rounds of 256x256 tiles (N 20480, K 4096, T
// 1000, the 64 of 80, us all / none / split: MXFP4 and bf16 x 171 / 144 / 134,
// MXFP8 x 103 / 93 / 82, MXFP8 weights 101 / 97 / 85). With two 128x128
// workgroups on a compute unit one's epilogue runs beside the other's loop. The
// times (ns) are fitted to T 65-8192, N 96-35840, K 128-4096 for each kernel; kv
// is the same bit for bit whatever the tile.
struct TileTimes {
  int big, big_k;     // a round of 256x256 tiles
  int full, full_k;   // a round of 128x128 tiles, two on a compute unit
  int half, half_k;   // the same, one on a compute unit
};

inline int big_columns(int64_t T, int64_t N, int K, const TileTimes& t) {
  const int64_t cus = dev_info().num_cus, ks = K / 128;
  const int64_t tt = (T + 255) / 256, tn = (N + 255) / 256, rounds = tn * tt / cus;
  const int64_t big = t.big + t.big_k * ks, full = t.full + t.full_k * ks, half = t.half + t.half_k * ks;
  auto small = [&](int64_t rows) {
    const int64_t n = ((rows + 127) / 128) * ((T + 127) / 128), last = n % (2 * cus);
    return n / (2 * cus) * full + (last > cus ? full : last > 0 ? half : 0);
  };
  int64_t best = (tn * tt + cus - 1) / cus * big, cols = tn;
  if (small(N) < best) best = small(N), cols = 0;
  const int64_t part = rounds * cus / tt, second_launch = 3500;
  if (rounds > 0 && part < tn && rounds * big + small(N - 256 * part) + second_launch < best) cols = part;
  return (int)cols;
}

inline hipError_t set_lds(const void* fn, int bytes) {
  return hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace

}  // namespace engram
