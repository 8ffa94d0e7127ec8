// Projection with MXFP4 weights for small batches (T <= 64): kv[T, N] =
// bf16(x . deq(W)^T), x bf16 (fp32 sums) or MXFP8 (fp32 but for runs of 8 k).
//
// W is e2m1 codes [N, K/2] with one E8M0 byte per row and 32 k [N, K/32] (OCP
// MX v1.0 MXFP4). With few tokens the product is a stream of the
// weight, here of 17/32 byte per weight: half of MXFP8's, a quarter of bf16's.
//
// A workgroup owns RT tiles of 16 W rows and all T tokens (NT tiles of 16);
// each of its waves takes a contiguous run of k steps of 128, and the waves'
// partial 16x16 tiles are summed through LDS in wave order. In a k step lane l
// holds row l%16 and, with g = l/16, the 16 bytes of k 32g .. 32g+31: exactly
// one scale group, so a fragment meets one scale byte.
//  * x bf16: v_cvt_scalef32_pk_bf16_fp4 turns a byte into two scaled bf16
//    (exact; of its fp32 scale operand it takes the exponent field, as E8M0:
//    0 is 2^-127, 255 NaN), and v_mfma_f32_16x16x32_bf16 number i (0..3) takes
//    each lane's word i, k 32g+8i .. 32g+8i+7 (the order of k inside a product
//    is free as long as both operands follow it), against x at that k.
//  * x MXFP8: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies the e2m1 codes as
//    they are with e4m3 codes. Lane layout (measured with one-hot operands and
//    distinct per-lane scales): the fp4 operand's 16 bytes are k 32g..32g+31 in
//    order; the fp8 operand's bytes 0..15 are k 16g.. and 16..31 are k 64+16g..;
//    lane group g's E8M0 byte scales k block [32g, 32g+32) of either. (Inside
//    the instruction a run of 8 k is summed in a window of 14 bits below its
//    largest product, the runs in fp32: the same as with MXFP8 weights.)
//
// What bounds it, and why everything goes through LDS: the vector cache
// answers one cache line per clock and lane quarter, so a fragment load
// straight from memory (16 rows, 16 bytes of each) costs 64 clocks per KiB and
// scale bytes as much again. Direct-to-LDS DMAs that walk the rows (16 rows x
// 64 bytes of W, 4 x 256 or 8 x 128 bytes of x) cost 8 to 16, and the
// workgroup's scale bytes are one contiguous run. The rings are private to a
// wave: it waits for its own DMAs only, no barrier in the loop.
//
// Measured (N 20480, K 2048, 22.3 MB of weight; graph replay, about 2.5 us of
// it an empty kernel's): x bf16, T 1 / 16 / 32 / 48 / 61 in 7.0 / 7.3 / 9.0 /
// 10.8 / 12.2 us (fragments straight from memory, T 1 / 16 / 32 / 61: 9.0 /
// 10.5 / 12.9 / 17), x MXFP8 6.2 / 6.4 / 7.7 / 8.8 / 9.8 us. Up to 16 tokens the
// weight's stream bounds it (5 TB/s past the launch). Beyond 32 two things are
// not told apart: 256 workgroups read x's 250 KB (bf16, T 61) each from L2, three
// times the weight's bytes, and a wave has one unit of x in flight (bf16: at K
// 2048 four trips to memory, one after the other).
#include <algorithm>

#include "common.h"
#include "gemv_fp4_dma.h"

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

struct Gemv4Args {
  const void* x;           // bf16 [T, K] or e4m3 codes [T, K]
  const uint8_t* xs;       // E8M0 [T, K/32] (MXFP8 x)
  const uint8_t* w;        // [N, K/2]
  const uint8_t* ws;       // [N, K/32]
  uint16_t* kv;
  int T, K, N;
};

// x moves in units of JG token tiles of one k step, UPS units a step (four bf16
// tiles, 16 KB, would leave LDS for 7 waves at most).
constexpr int f4_jg(bool a8, int nt) { return !a8 && nt == 4 ? 2 : nt; }
constexpr int f4_ups(bool a8, int nt) { return nt / f4_jg(a8, nt); }
// W steps in the ring when XS units of x are (two units a step: one at a time)
constexpr int f4_dw(bool a8, int nt, int xs) { return f4_ups(a8, nt) == 1 ? xs : 1; }
constexpr int f4_xunit(bool a8, int nt) { return f4_jg(a8, nt) * (a8 ? 2048 : 4096); }
constexpr int f4_wave_bytes(bool a8, int rt, int nt, int xs) {
  return f4_dw(a8, nt, xs) * rt * 1024 + xs * f4_xunit(a8, nt);
}
constexpr int f4_up(int v, int m) { return (v + m - 1) / m * m; }
// LDS: W's scale bytes | x's scale bytes | a ring per wave; afterwards the
// waves' partial tiles.
constexpr int f4_lds(bool a8, int rt, int nt, int waves, int xs, int kb) {
  const int in = f4_up(16 * rt * kb, 1024) + (a8 ? f4_up(16 * nt * kb, 256) : 0) +
                 waves * f4_wave_bytes(a8, rt, nt, xs);
  const int red = waves * rt * nt * 1024;
  return in > red ? in : red;
}

template <bool A8, int RT, int NT, int WAVES, int XS, bool SWAP>
__global__ __launch_bounds__(WAVES * 64) void gemv_mxfp4_kernel(
    const uint8_t* __restrict__ x, const uint8_t* __restrict__ xs, int T, int K, const uint8_t* __restrict__ w,
    const uint8_t* __restrict__ ws, int N, uint16_t* __restrict__ kv) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  constexpr int JG = f4_jg(A8, NT), UPS = f4_ups(A8, NT), DW = f4_dw(A8, NT, XS);
  constexpr int XUNIT = f4_xunit(A8, NT), XI = XUNIT / 1024;   // DMAs of a unit of x
  static_assert(UPS == 1 || XS == 1, "ring schedule");
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * RT, rows = min(16 * RT, N - n0);
  const int g = lane >> 4, r = lane & 15;
  const int nsteps = K / 128, kb = K / 32;
  const int per = (nsteps + WAVES - 1) / WAVES;
  const int s0 = min(wave * per, nsteps), units = (min(s0 + per, nsteps) - s0) * UPS;

  const int xsl = f4_up(16 * RT * kb, 1024);                     // x's scale bytes
  const int ring = xsl + (A8 ? f4_up(16 * NT * kb, 256) : 0) + wave * f4_wave_bytes(A8, RT, NT, XS);
  const int xring = ring + DW * RT * 1024;

  // Range-checked DMAs: a lane's vector offset is its row and piece, the step
  // rides in the scalar offset. A row past N or a token past T is past the
  // range whatever the step and fills zeros.
  const int wpitch = K / 2, xpitch = A8 ? K : K * 2;
  const rsrc_t rw = make_rsrc(w + (int64_t)n0 * wpitch, (uint32_t)rows * (uint32_t)wpitch);
  const rsrc_t rx = make_rsrc(x, (uint32_t)T * (uint32_t)xpitch);

  // Scale bytes: contiguous over the workgroup's rows (and over x's tokens,
  // whose count of bytes is a multiple of 4 only). A step's read takes one
  // word of each of 16 rows, kb bytes apart. SWAP (kb % 128 == 0: those words
  // share one or two banks of 16): the 16-byte pieces of row r are swapped by
  // 3 or 4 bits of r, for 8 or 16 | kb / 16, which puts them on distinct banks.
  {
    const rsrc_t rs = make_rsrc(ws + (int64_t)n0 * kb, (uint32_t)rows * (uint32_t)kb);
    for (int q = wave; q * 1024 < 16 * RT * kb; q += WAVES) {
      const uint32_t vo = fp4::s_source(SWAP, (uint32_t)(q * 1024 + lane * 16), (uint32_t)kb);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rs, (lds_ptr_t)(lds + q * 1024), 16, vo, 0, 0, 0);
    }
    if constexpr (A8) {
      const rsrc_t rxs = make_rsrc(xs, (uint32_t)T * (uint32_t)kb);
      for (int q = wave; q * 256 < 16 * NT * kb; q += WAVES)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rxs, (lds_ptr_t)(lds + xsl + q * 256), 4,
                                                 (uint32_t)(q * 256 + lane * 4), 0, 0, 0);
    }
  }

  // the DMAs' lane offsets and the fragments' LDS addresses: gemv_fp4_dma.h
  auto issue = [&](int u) {   // unit u of this wave: W with a step's first unit, then x
    const int s = s0 + u / UPS, j0 = u % UPS * JG;
    if (j0 == 0) {
      const int slot = ring + (s - s0) % DW * (RT * 1024);
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(lds + slot + rt * 1024), 16,
                                                 fp4::w_voffset(lane, rt, wpitch), s * fp4::kWStep, 0, 0);
    }
    const int slot = xring + u % XS * XUNIT;
#pragma unroll
    for (int i = 0; i < XI; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rx, (lds_ptr_t)(lds + slot + i * 1024), 16,
                                               fp4::x_voffset(A8, lane, j0 * 16, i, xpitch), s * fp4::x_step(A8), 0, 0);
  };

  f32x4 acc[RT][NT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  // DMAs of the units after the one at hand that may still fly
  constexpr int AHEAD = (XS - 1) * (RT + XI);
  for (int u = 0; u < XS; ++u)
    if (u < units) issue(u);
  // the scale bytes of all waves
  if (units >= XS) wait_vm<AHEAD + RT + XI>();
  else wait_vm<0>();
  bare_barrier();

  auto multiply = [&](int u, int p) {   // p: u % UPS, static
    const int s = s0 + u / UPS;
    const char* wl = lds + ring + (s - s0) % DW * (RT * 1024) + fp4::w_read(r, g);
    const char* xl = lds + xring + u % XS * XUNIT;
    const uint8_t* sl = reinterpret_cast<const uint8_t*>(lds) + fp4::s_read(SWAP, (uint32_t)r, (uint32_t)(s * 4), (uint32_t)kb) + g;
    i32x4 wv[RT];
    uint32_t sc[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      wv[rt] = *reinterpret_cast<const i32x4*>(wl + rt * 1024);
      sc[rt] = sl[rt * 16 * kb];
    }
    if constexpr (A8) {
#pragma unroll
      for (int j = 0; j < JG; ++j) {
        const i32x4 lo = *reinterpret_cast<const i32x4*>(xl + j * 2048 + fp4::x_read(true, r, g));
        const i32x4 hi = *reinterpret_cast<const i32x4*>(xl + j * 2048 + fp4::x_read(true, r, 4 + g));
        const int xsc = sl[xsl + j * 16 * kb];
        const i32x8 xb = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          // fp4: the first four words
          const i32x8 wa = __builtin_shufflevector(wv[rt], wv[rt], 0, 1, 2, 3, 0, 1, 2, 3);
          acc[rt][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc[rt][j], 4, 0, 0, (int)sc[rt], 0,
                                                                       xsc);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf16x8_t xb[JG];
#pragma unroll
        for (int j = 0; j < JG; ++j)
          xb[j] = *reinterpret_cast<const bf16x8_t*>(xl + j * 4096 + fp4::x_read(false, r, 4 * g + i));
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float scale = __uint_as_float(sc[rt] << 23);
          const uint32_t w4 = (uint32_t)wv[rt][i];
          const uint4 wb = make_uint4(fp4_pair_to_bf16<0>(w4, scale), fp4_pair_to_bf16<1>(w4, scale),
                                      fp4_pair_to_bf16<2>(w4, scale), fp4_pair_to_bf16<3>(w4, scale));
#pragma unroll
          for (int j = 0; j < JG; ++j)
            acc[rt][p * JG + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wb), xb[j],
                                                                         acc[rt][p * JG + j], 0, 0, 0);
        }
      }
    }
  };

  for (int u0 = 0; u0 < units; u0 += UPS) {
#pragma unroll
    for (int p = 0; p < UPS; ++p) {
      const int u = u0 + p;
      if (u + XS <= units) wait_vm<AHEAD>();   // every unit ahead has been issued
      else wait_vm<0>();
      multiply(u, p);
      if (u + XS < units) {
        wait_lgkm0();   // this unit's reads are done before its slots are filled again
        issue(u + XS);
      }
    }
  }

  wait_lgkm0();
  bare_barrier();   // every wave is done with its ring (and has no DMA left)
  f32x4* red = reinterpret_cast<f32x4*>(lds);
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * RT * NT + rt * NT + j) * 64 + lane] = acc[rt][j];
  __syncthreads();
  // thread (tile pair, lane) sums the waves' partials in wave order; C lane l
  // holds rows 4*(l/16)+i of the row tile, token l%16
  for (int idx = tid; idx < RT * NT * 64; idx += WAVES * 64) {
    const int pair = idx >> 6, l = idx & 63;
    const int rt = pair / NT, j = pair - rt * NT;
    f32x4 sum = red[pair * 64 + l];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) {
      const f32x4 p = red[(v * RT * NT + pair) * 64 + l];
      sum[0] += p[0]; sum[1] += p[1]; sum[2] += p[2]; sum[3] += p[3];
    }
    const int t = j * 16 + (l & 15);
    const int n = n0 + rt * 16 + 4 * (l >> 4);
    if (t < T && n < N) {   // N % 4 == 0: the four rows are in or out together
      uint2 o;
      o.x = cvt_pk_bf16(sum[0], sum[1]);
      o.y = cvt_pk_bf16(sum[2], sum[3]);
      *reinterpret_cast<uint2*>(kv + (int64_t)t * N + n) = o;
    }
  }
}

template <bool A8, int RT, int NT, int WAVES, int XS>
hipError_t f4_launch(const Gemv4Args& a, hipStream_t s) {
  const int lds = f4_lds(A8, RT, NT, WAVES, XS, a.K / 32);
  // swapped scale pieces: N 20480, K 4096, bf16 x, T 1 / 61 11.5 / 20.7 ->
  // 10.7 / 18.5 us (at K 2048 and with MXFP8 x the index work costs as much)
  const bool swap = !A8 && a.K % 4096 == 0;
  const auto fn = swap ? gemv_mxfp4_kernel<A8, RT, NT, WAVES, XS, !A8> : gemv_mxfp4_kernel<A8, RT, NT, WAVES, XS, false>;
  if (lds > 64 * 1024) {   // above the default limit
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((a.N + 16 * RT - 1) / (16 * RT)), dim3(WAVES * 64), lds, s, (const uint8_t*)a.x, a.xs,
                     a.T, a.K, a.w, a.ws, a.N, a.kv);
  return hipGetLastError();
}

// Little x (up to 16 tokens, 32 in MXFP8): small workgroups, several on a
// compute unit, hide each other's latencies: 4 waves, one step in flight, two
// row tiles (N 20480, K 2048, T 16, bf16 / MXFP8 x: 7.3 / 6.3 us; 8 waves of
// five row tiles 7.6 / 6.7, one row tile 8.7 / 6.8). With fewer row tiles
// than compute units, one tile over 8 waves (N 2560: 3.1 us against 3.4).
template <bool A8, int NT>
hipError_t f4_small(const Gemv4Args& a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, cus = dev_info().num_cus, kb = a.K / 32;
  if (tiles >= 2 * cus && f4_lds(A8, 2, NT, 4, 1, kb) <= kLds) return f4_launch<A8, 2, NT, 4, 1>(a, s);
  if (tiles <= cus && f4_lds(A8, 1, NT, 8, 1, kb) <= kLds) return f4_launch<A8, 1, NT, 8, 1>(a, s);
  return f4_launch<A8, 1, NT, 4, 1>(a, s);
}

// More x: one workgroup fills a compute unit's LDS, and each reads all of x,
// so as few as fill the compute units once: the least row-tile count that
// does, at most 5 (N 20480, K 2048, T 61, bf16 x: 12.2 us, two tiles in
// three rounds 19), less where the scale bytes of a long K do not fit.
template <bool A8, int NT, int WAVES, int XS>
hipError_t f4_large(const Gemv4Args& a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, cus = dev_info().num_cus, kb = a.K / 32;
  int rt = std::min(5, (tiles + cus - 1) / cus);
  while (rt > 1 && f4_lds(A8, rt, NT, WAVES, XS, kb) > kLds) --rt;
  switch (rt) {
    case 5: return f4_launch<A8, 5, NT, WAVES, XS>(a, s);
    case 4: return f4_launch<A8, 4, NT, WAVES, XS>(a, s);
    case 3: return f4_launch<A8, 3, NT, WAVES, XS>(a, s);
    case 2: return f4_launch<A8, 2, NT, WAVES, XS>(a, s);
    default: return f4_launch<A8, 1, NT, WAVES, XS>(a, s);
  }
}

}  // namespace

bool gemv_mxfp4_supported(int64_t T, int K, bool x_mxfp8) {
  if (T < 1 || T > kGemvMaxT) return false;
  // the smallest instantiation's LDS (past 32 tokens of MXFP8 x the four-tile one's,
  // though up to 48 run three tiles, which K 53248 would fit)
  const int kb = std::min(K, 1 << 20) / 32;
  if (x_mxfp8) return (T <= 16 ? f4_lds(true, 1, 1, 4, 1, kb) : T <= 32 ? f4_lds(true, 1, 2, 4, 1, kb)
                                                                        : f4_lds(true, 1, 4, 4, 2, kb)) <= kLds;
  return (T <= 16 ? f4_lds(false, 1, 1, 4, 1, kb) : T <= 32 ? f4_lds(false, 1, 2, 8, 1, kb)
                                                            : f4_lds(false, 1, 4, 8, 1, kb)) <= kLds;
}

hipError_t launch_gemv_mxfp4(const void* x, const uint8_t* xs, int64_t T, int K, const void* w, const uint8_t* ws,
                             int N, void* kv, hipStream_t s) {
  const Gemv4Args a{x, xs, (const uint8_t*)w, ws, (uint16_t*)kv, (int)T, K, N};
  if (xs)
    return T <= 16 ? f4_small<true, 1>(a, s) : T <= 32 ? f4_small<true, 2>(a, s)
         : T <= 48 ? f4_large<true, 3, 4, 2>(a, s) : f4_large<true, 4, 4, 2>(a, s);
  if (T <= 16) return f4_small<false, 1>(a, s);
  if (T <= 32) return f4_large<false, 2, 8, 1>(a, s);
  // three tiles in one unit a step: T 48 12.2 -> 10.8 us (MXFP8 x 9.3 -> 8.8)
  if (T <= 48 && f4_lds(false, 1, 3, 8, 1, K / 32) <= kLds) return f4_large<false, 3, 8, 1>(a, s);
  return f4_large<false, 4, 8, 1>(a, s);
}

}  // namespace engram
