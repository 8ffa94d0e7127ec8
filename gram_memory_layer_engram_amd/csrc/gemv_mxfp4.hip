// Projection with MXFP4 weights for small batches (T <= 64): kv[T, N] =
// bf16(x . deq(W)^T), x bf16 or MXFP8, fp32 accumulation.
//
// W is e2m1 codes [N, K/2] with one E8M0 byte per row and 32 k [N, K/32] (OCP
// MX v1.0 MXFP4). With few tokens the product is a stream of the weight
// ("vllm.models.deepseek_v41.amd.mono.attention.gemv": weight loads in flight
// before the activations, split over k), here of 17/32 byte per weight: half
// of MXFP8's, a quarter of bf16's.
//
// Layout, as in the other decode GEMVs: a workgroup of 8 waves owns RT tiles
// of 16 W rows and all T tokens (NT tiles of 16); wave w takes k steps of
// 128, and the waves' partial 16x16 tiles are summed through LDS in wave
// order. In a k step lane l holds row l%16 and, with g = l/16, the 16 bytes
// of k 32g .. 32g+31: exactly one scale group, so a lane's 16-byte load meets
// one scale byte.
//  * x bf16: v_cvt_scalef32_pk_bf16_fp4 turns a byte into two scaled bf16
//    (exact), and v_mfma_f32_16x16x32_bf16 number i (0..3) takes each lane's
//    word i, k 32g+8i .. 32g+8i+7 (the order of k inside a product is free as
//    long as both operands follow it), against the 16 bytes of x at that k.
//  * x MXFP8: v_mfma_scale_f32_16x16x128_f8f6f4 multiplies the e2m1 codes as
//    they are with e4m3 codes. Lane layout (measured with one-hot operands and
//    distinct per-lane scales): the fp4 operand's 16 bytes are k 32g..32g+31 in
//    order; the fp8 operand's bytes 0..15 are k 16g.. and 16..31 are k 64+16g..;
//    lane group g's E8M0 byte scales k block [32g, 32g+32) of either.
#include "common.h"
#include "fp8_table.h"

namespace engram {

namespace {

constexpr int F4_WAVES = 8;
constexpr int F4_THREADS = F4_WAVES * 64;

constexpr int f4_lds(int rt, int nt) { return F4_WAVES * rt * nt * 64 * 16; }

struct Gemv4Args {
  const void* x;           // bf16 [T, K] or e4m3 codes [T, K]
  const uint8_t* xs;       // E8M0 [T, K/32] (MXFP8 x)
  const uint8_t* w;        // [N, K/2]
  const uint8_t* ws;       // [N, K/32]
  uint16_t* kv;
  int T, K, N;
};

// SPW: k steps of one wave per pass; K past 8 * SPW steps takes more passes.
template <bool A8, int RT, int NT, int SPW>
__global__ __launch_bounds__(F4_THREADS) void gemv_mxfp4_kernel(const Gemv4Args a) {
  extern __shared__ __attribute__((aligned(1024))) char lds[];
  f32x4* red = reinterpret_cast<f32x4*>(lds);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16 * RT;
  const int g = lane >> 4, r = lane & 15;
  const int nsteps = a.K / 128, kb = a.K / 32;

  // a row past N reads row N-1, a token past T reads token 0: their products
  // only feed outputs that are not stored
  const uint8_t* wrow[RT];
  const uint8_t* srow[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int64_t n = min(n0 + rt * 16 + r, a.N - 1);
    wrow[rt] = a.w + n * (a.K / 2) + 16 * g;
    srow[rt] = a.ws + n * kb + g;
  }
  const uint8_t* xrow[NT];
  const uint8_t* xsrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t t = j * 16 + r < a.T ? j * 16 + r : 0;
    xrow[j] = (const uint8_t*)a.x + (A8 ? t * a.K + 16 * g : t * a.K * 2 + 64 * g);
    xsrow[j] = A8 ? a.xs + t * kb + g : nullptr;
  }

  f32x4 acc[RT][NT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[rt][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  for (int base = wave * SPW; base < nsteps; base += F4_WAVES * SPW) {
    // all of the pass's weight loads first, then x; the bounds tests are
    // uniform and keep the loads from being moved next to their uses
    uint4 wv[RT][SPW];
    uint32_t sc[RT][SPW];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        wv[rt][s] = make_uint4(0, 0, 0, 0);
        sc[rt][s] = 0;
        if (base + s < nsteps) {
          wv[rt][s] = *reinterpret_cast<const uint4*>(wrow[rt] + (int64_t)(base + s) * 64);
          sc[rt][s] = srow[rt][(base + s) * 4];
        }
      }
    if constexpr (A8) {
      uint4 lo[NT][SPW], hi[NT][SPW];
      uint32_t xsc[NT][SPW];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int s = 0; s < SPW; ++s) {
          lo[j][s] = hi[j][s] = make_uint4(0, 0, 0, 0);
          xsc[j][s] = 0;
          if (base + s < nsteps) {
            lo[j][s] = *reinterpret_cast<const uint4*>(xrow[j] + (int64_t)(base + s) * 128);
            hi[j][s] = *reinterpret_cast<const uint4*>(xrow[j] + (int64_t)(base + s) * 128 + 64);
            xsc[j][s] = xsrow[j][(base + s) * 4];
          }
        }
#pragma unroll
      for (int s = 0; s < SPW; ++s) {
        if (base + s >= nsteps) break;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const i32x8 xb = __builtin_shufflevector(__builtin_bit_cast(i32x4, lo[j][s]),
                                                   __builtin_bit_cast(i32x4, hi[j][s]), 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const i32x4 wq = __builtin_bit_cast(i32x4, wv[rt][s]);
            const i32x8 wa = __builtin_shufflevector(wq, wq, 0, 1, 2, 3, 0, 1, 2, 3);
            acc[rt][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, xb, acc[rt][j], 4, 0, 0,
                                                                         (int)sc[rt][s], 0, (int)xsc[j][s]);
          }
        }
      }
    } else {
      // x in units of JG token tiles of one step, a ring of them in flight
      constexpr int JG = NT < 2 ? NT : 2, UPS = NT / JG, UNITS = SPW * UPS;
      constexpr int RING = UNITS < 3 ? UNITS : 3;
      uint4 xv[RING][JG][4];
      auto load_x = [&](int u) {
        const int s = u / UPS, j0 = (u % UPS) * JG;
        if (base + s < nsteps) {
#pragma unroll
          for (int j = 0; j < JG; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              xv[u % RING][j][i] =
                  *reinterpret_cast<const uint4*>(xrow[j0 + j] + (int64_t)(base + s) * 256 + 16 * i);
        }
      };
#pragma unroll
      for (int u = 0; u < RING; ++u) load_x(u);
#pragma unroll
      for (int u = 0; u < UNITS; ++u) {
        const int s = u / UPS, j0 = (u % UPS) * JG;
        if (base + s >= nsteps) break;
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float scale = e8m0_to_f32(sc[rt][s]);
          const uint32_t w4[4] = {wv[rt][s].x, wv[rt][s].y, wv[rt][s].z, wv[rt][s].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 wb = make_uint4(fp4_pair_to_bf16<0>(w4[i], scale), fp4_pair_to_bf16<1>(w4[i], scale),
                                        fp4_pair_to_bf16<2>(w4[i], scale), fp4_pair_to_bf16<3>(w4[i], scale));
#pragma unroll
            for (int j = 0; j < JG; ++j)
              acc[rt][j0 + j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  __builtin_bit_cast(bf16x8_t, wb), __builtin_bit_cast(bf16x8_t, xv[u % RING][j][i]),
                  acc[rt][j0 + j], 0, 0, 0);
          }
        }
        if (u + RING < UNITS) load_x(u + RING);
      }
    }
  }

#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(wave * RT * NT + rt * NT + j) * 64 + lane] = acc[rt][j];
  __syncthreads();
  // thread (tile pair, lane) sums the waves' partials in wave order; C lane l
  // holds rows 4*(l/16)+i of the row tile, token l%16
  for (int idx = tid; idx < RT * NT * 64; idx += F4_THREADS) {
    const int pair = idx >> 6, l = idx & 63;
    const int rt = pair / NT, j = pair - rt * NT;
    f32x4 sum = red[pair * 64 + l];
#pragma unroll
    for (int v = 1; v < F4_WAVES; ++v) {
      const f32x4 p = red[(v * RT * NT + pair) * 64 + l];
      sum[0] += p[0]; sum[1] += p[1]; sum[2] += p[2]; sum[3] += p[3];
    }
    const int t = j * 16 + (l & 15);
    const int n = n0 + rt * 16 + 4 * (l >> 4);
    if (t < a.T && n < a.N) {   // N % 4 == 0: the four rows are in or out together
      uint2 o;
      o.x = cvt_pk_bf16(sum[0], sum[1]);
      o.y = cvt_pk_bf16(sum[2], sum[3]);
      *reinterpret_cast<uint2*>(a.kv + (int64_t)t * a.N + n) = o;
    }
  }
}

template <bool A8, int RT, int NT, int SPW>
hipError_t f4_launch(const Gemv4Args& a, hipStream_t s) {
  constexpr int lds = f4_lds(RT, NT);
  const auto fn = gemv_mxfp4_kernel<A8, RT, NT, SPW>;
  if constexpr (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute((const void*)fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(fn, dim3((a.N + 16 * RT - 1) / (16 * RT)), dim3(F4_THREADS), lds, s, a);
  return hipGetLastError();
}

// Two steps a wave and pass once K has them (2048 and up: all of a row tile's
// bytes of a pass in flight at once), else one.
template <bool A8, int RT, int NT>
hipError_t f4_spw(const Gemv4Args& a, hipStream_t s) {
  return a.K / 128 > F4_WAVES ? f4_launch<A8, RT, NT, 2>(a, s) : f4_launch<A8, RT, NT, 1>(a, s);
}

// The largest row-tile count that still gives every compute unit a workgroup:
// each re-reads all of x from L2.
template <bool A8, int NT>
hipError_t f4_rt(const Gemv4Args& a, hipStream_t s) {
  const int tiles = (a.N + 15) / 16, cus = dev_info().num_cus;
  if (tiles >= 5 * cus) return f4_spw<A8, 5, NT>(a, s);
  if (tiles >= 4 * cus) return f4_spw<A8, 4, NT>(a, s);
  if (tiles >= 2 * cus) return f4_spw<A8, 2, NT>(a, s);
  return f4_spw<A8, 1, NT>(a, s);
}

template <bool A8>
hipError_t f4_nt(const Gemv4Args& a, hipStream_t s) {
  if (a.T <= 16) return f4_rt<A8, 1>(a, s);
  if (a.T <= 32) return f4_rt<A8, 2>(a, s);
  return f4_rt<A8, 4>(a, s);
}

}  // namespace

hipError_t launch_gemv_mxfp4(const void* x, const uint8_t* xs, int64_t T, int K, const void* w, const uint8_t* ws,
                             int N, void* kv, hipStream_t s) {
  const Gemv4Args a{x, xs, (const uint8_t*)w, ws, (uint16_t*)kv, (int)T, K, N};
  return xs ? f4_nt<true>(a, s) : f4_nt<false>(a, s);
}

}  // namespace engram
