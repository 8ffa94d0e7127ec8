// Host model of the int8 kernels' global -> LDS DMAs (csrc/gemv_int8_dma.h, and
// csrc/gemm_dma.h on rows of K bytes with K % 16 == 0): for ragged rows, tokens and K
// every lane and DMA of every step is evaluated with the kernels' own functions. A
// vector offset must lie a whole piece inside the range or past it; the LDS image is
// filled with the global byte each DMA would bring (or "zero"), and every fragment
// read must find the bytes of its row and k, or zeros (x past its row's end). Bank
// conflicts: the eight rows that a 128-byte LDS cycle serves must not collide.
// Prints one summary line; exit status 0 when every check passes.
#include "../gram_memory_layer_engram_amd/csrc/gemm_dma.h"
#include "../gram_memory_layer_engram_amd/csrc/gemv_int8_dma.h"

#include <cstdint>
#include <cstdio>
#include <vector>

namespace {

namespace i8 = engram::i8;
namespace dma = engram::dma;
long long g_checks = 0;
int g_fail = 0;

void expect(bool ok, const char* what, long long a, long long b, long long c) {
  ++g_checks;
  if (ok) return;
  if (g_fail++ < 20) std::printf("FAIL %s: %lld %lld %lld\n", what, a, b, c);
}

// The global byte that a lane's 16 bytes come from, or -1 for zeros.
long long source(uint32_t vo, int rows, int K) {
  const uint64_t range = (uint64_t)rows * K;
  const bool inside = (uint64_t)vo + 16 <= range, outside = (uint64_t)vo >= range;
  expect(inside || outside, "straddles the range end", vo, (long long)range, K);
  expect(vo < 0x80000000u, "offset >= 2^31", vo, 0, 0);
  return inside ? (long long)vo : -1;
}

// Rows [0, rows) of `tiles` tiles of 16, step s: as the register kernel fetches W
// (no check of the row's end) and as the slice kernel fetches both (`tail`).
void gemv(int tiles, int rows, int K, bool tail_check) {
  const int nk = (K + i8::kStep - 1) / i8::kStep;
  for (int s = 0; s <= nk; ++s) {   // nk: a step that does not exist
    std::vector<long long> img(tiles * 128);
    for (int q = 0; q < 2 * tiles; ++q)
      for (int lane = 0; lane < 64; ++lane) {
        uint32_t vo;
        if (tail_check) {
          const bool tail = (uint32_t)(nk - 1) * i8::kStep + i8::piece_of(lane) >= (uint32_t)K;
          const uint32_t kofs = s < nk ? (uint32_t)s * i8::kStep : i8::kOob;
          vo = i8::voffset(lane, q, 0u, (uint32_t)K) + (tail && s == nk - 1 ? i8::kOob : kofs);
        } else {
          vo = i8::voffset(lane, q, s * i8::kStep < K ? (uint32_t)s * i8::kStep : i8::kOob, (uint32_t)K);
        }
        img[q * 64 + lane] = source(vo, rows, K);
      }
    for (int t = 0; t < tiles; ++t)
      for (int r = 0; r < 16; ++r)
        for (int p = 0; p < 8; ++p) {
          const int row = t * 16 + r, k = s * i8::kStep + 16 * p;
          const long long got = img[t * 128 + i8::read(r, p) / 16], at = (long long)row * K + k;
          if (row < rows && k < K) expect(got == at, "fragment", row, k, got);
          // x past its end has to be zeros; W there only has to be readable
          else if (tail_check || row >= rows || s == nk) expect(got == -1, "not zeros past the end", row, k, got);
        }
  }
}

void gemm(int tile, int rows, int K) {
  const uint32_t oob = (uint32_t)tile * (uint32_t)K;
  const int nk = (K + 127) / 128;
  for (int d = 0; d <= nk; ++d) {
    const uint32_t kofs = d < nk ? (uint32_t)d * 128 : oob;
    std::vector<long long> img(tile * 8, -2);
    for (int wave = 0; wave < 4; ++wave)
      for (int i = 0; i < tile / 32; ++i)
        for (int lane = 0; lane < 64; ++lane) {
          const dma::Lane l = dma::lane_of(wave, lane, (uint32_t)K);
          img[(wave + 4 * i) * 64 + lane] = source(dma::voffset(l, i, kofs, (uint32_t)K, oob, K % 128 != 0), rows, K);
        }
    for (int row = 0; row < tile; ++row)
      for (int p = 0; p < 8; ++p) {
        const long long got = img[row * 8 + (p ^ dma::swizzle(row))];
        const int k = d * 128 + 16 * p;
        expect(got == (row < rows && k < K ? (long long)row * K + k : -1), "GEMM fragment", row, k, got);
      }
  }
}

}  // namespace

int main() {
  for (int K : {16, 48, 112, 128, 144, 1040, 2048, 131056}) {
    for (int rows : {1, 7, 16}) gemv(1, rows, K, false), gemv(1, rows, K, true);
    for (int rows : {33, 48}) gemv(3, rows, K, false), gemv(3, rows, K, true);
    if (K <= 2048)
      for (int rows : {100, 112, 128}) gemv(8, rows, K, true), gemm(128, rows, K), gemm(256, rows + 100, K);
  }
  for (int p = 0; p < 8; ++p)
    for (int r0 = 0; r0 < 16; r0 += 8) {
      int seen = 0;
      for (int r = r0; r < r0 + 8; ++r) seen |= 1 << (i8::read(r, p) / 16 % 8);
      expect(seen == 0xff, "bank conflict", p, r0, seen);
    }
  std::printf("%lld checks, %d failures\n", g_checks, g_fail);
  return g_fail ? 1 : 0;
}
