// Host model of the MXFP4 kernels' global -> LDS DMAs.
//
// GEMV (csrc/gemv_fp4_dma.h): for ragged rows and tokens, every lane and DMA
// of every step is evaluated with the kernel's own functions, the LDS image is
// filled with the global byte each DMA would bring (or "zero"), and every
// fragment and scale read is checked to find exactly its bytes. A lane's
// vector offset must lie a whole piece inside the range or past it, and with
// the unchecked scalar offset an in-range lane must stay inside its own row.
// Bank conflicts: the eight rows a 128-byte LDS cycle serves must not collide.
//
// GEMM (csrc/gemm_dma.h on 4-bit row pitches): chunks of 128 bytes of W rows of
// K / 2 bytes, tiles of 256 and 128 rows.
// Prints one summary line; exit status 0 when every check passes.
#include "../gram_memory_layer_engram_amd/csrc/gemm_dma.h"
#include "../gram_memory_layer_engram_amd/csrc/gemv_fp4_dma.h"

#include <cstdint>
#include <cstdio>
#include <vector>

namespace {

namespace fp4 = engram::fp4;
long long g_checks = 0;
int g_fail = 0;

void expect(bool ok, const char* what, long long a, long long b, long long c) {
  ++g_checks;
  if (ok) return;
  if (g_fail++ < 20) std::printf("FAIL %s: %lld %lld %lld\n", what, a, b, c);
}

// One DMA of 64 lanes into img (16-byte pieces, value = global byte or -1):
// rows rows of pitch bytes, each lane moving 16 bytes of step `step`.
void dma(std::vector<long long>& img, int lds_piece, int lane, uint32_t vo, uint32_t so, int rows, int pitch,
         int step_bytes) {
  const uint64_t range = (uint64_t)rows * pitch;
  const bool inside = (uint64_t)vo + 16 <= range, outside = (uint64_t)vo >= range;
  expect(inside || outside, "straddles the range end", vo, range, pitch);
  expect(vo < 0x80000000u, "offset >= 2^31", vo, 0, 0);
  if (inside) {
    const uint64_t at = (uint64_t)vo + so;
    expect(vo % pitch + 16 <= (uint32_t)step_bytes, "piece outside its step", vo, pitch, step_bytes);
    expect(at / pitch == vo / pitch && at % pitch + 16 <= (uint64_t)pitch, "leaves its row", vo, so, pitch);
    img[lds_piece + lane] = (long long)at;
  } else {
    img[lds_piece + lane] = -1;
  }
}

void gemv_w(int rt_count, int rows, int K) {
  const int pitch = K / 2;
  for (int s = 0; s < K / 128; ++s) {
    std::vector<long long> img(rt_count * 64);
    for (int rt = 0; rt < rt_count; ++rt)
      for (int lane = 0; lane < 64; ++lane)
        dma(img, rt * 64, lane, fp4::w_voffset(lane, rt, pitch), (uint32_t)(s * fp4::kWStep), rows, pitch, fp4::kWStep);
    for (int rt = 0; rt < rt_count; ++rt)
      for (int r = 0; r < 16; ++r)
        for (int g = 0; g < 4; ++g) {
          const int row = rt * 16 + r;
          const long long want = row < rows ? (long long)row * pitch + s * 64 + 16 * g : -1;
          expect(img[rt * 64 + fp4::w_read(r, g) / 16] == want, "W fragment", row, s, g);
        }
  }
  for (int g = 0; g < 4; ++g)
    for (int r0 = 0; r0 < 16; r0 += 8) {
      int seen = 0;
      for (int r = r0; r < r0 + 8; ++r) seen |= 1 << (fp4::w_read(r, g) / 16 % 8);
      expect(seen == 0xff, "W bank conflict", g, r0, seen);
    }
}

void gemv_x(bool a8, int tiles, int T, int K) {
  const int pitch = a8 ? K : 2 * K, step = fp4::x_step(a8), per_tile = step * 16 / 1024;
  for (int s = 0; s < K / 128; ++s)
    for (int j = 0; j < tiles; ++j) {
      std::vector<long long> img(per_tile * 64);
      for (int i = 0; i < per_tile; ++i)
        for (int lane = 0; lane < 64; ++lane)
          dma(img, i * 64, lane, fp4::x_voffset(a8, lane, j * 16, i, pitch), (uint32_t)(s * step), T, pitch, step);
      for (int r = 0; r < 16; ++r)
        for (int p = 0; p < step / 16; ++p) {
          const int t = j * 16 + r;
          const long long want = t < T ? (long long)t * pitch + s * step + 16 * p : -1;
          expect(img[fp4::x_read(a8, r, p) / 16] == want, "x fragment", t, s, p);
        }
    }
  for (int p = 0; p < step / 16; ++p)
    for (int r0 = 0; r0 < 16; r0 += 8) {
      int seen = 0;
      for (int r = r0; r < r0 + 8; ++r) seen |= 1 << (fp4::x_read(a8, r, p) / 16 % 8);
      expect(seen == 0xff, "x bank conflict", p, r0, seen);
    }
}

void scales(int rt_count, int rows, uint32_t kb) {
  for (int swap = 0; swap < 2; ++swap) {
    if (swap && kb % 128 != 0) continue;
    const uint64_t range = (uint64_t)rows * kb;
    const uint32_t n = (uint32_t)(16 * rt_count) * kb, up = (n + 1023) / 1024 * 1024;
    std::vector<long long> img(up);
    for (uint32_t ofs = 0; ofs < up; ofs += 16) {
      const uint32_t vo = fp4::s_source(swap, ofs, kb);
      expect((uint64_t)vo + 16 <= range || vo >= range, "scales straddle the range end", vo, range, kb);
      for (int b = 0; b < 16; ++b) img[ofs + b] = (uint64_t)vo + 16 <= range ? (long long)vo + b : -1;
    }
    for (uint32_t row = 0; row < (uint32_t)(16 * rt_count); ++row)
      for (uint32_t s4 = 0; s4 < kb; s4 += 4)
        for (uint32_t g = 0; g < 4; ++g) {
          const long long want = (int)row < rows ? (long long)row * kb + s4 + g : -1;
          // the kernel reads tile row r and adds rt * 16 * kb: a multiple of 16 rows leaves the swap as it is
          const uint32_t at = fp4::s_read(swap, row % 16, s4, kb) + row / 16 * 16 * kb + g;
          expect(img[at] == want, "scale byte", row, s4, g);
        }
    if (swap)
      for (uint32_t s4 = 0; s4 < kb; s4 += 4) {
        uint64_t banks = 0;
        for (uint32_t r = 0; r < 16; ++r) banks |= 1ull << (fp4::s_read(true, r, s4, kb) / 4 % 64);
        expect(__builtin_popcountll(banks) == 16, "scale bank conflict", kb, s4, __builtin_popcountll(banks));
      }
  }
}

// A W operand of the tiled GEMM: tiles of tile_rows rows of K / 2 bytes.
void gemm_w(int total, int K, int tile_rows) {
  const uint32_t pitch = (uint32_t)K / 2, oob = (uint32_t)tile_rows * pitch;
  for (int row0 = 0; row0 < total; row0 += tile_rows) {
    const int rows = total - row0 < tile_rows ? total - row0 : tile_rows;
    const uint64_t range = (uint64_t)rows * pitch;
    for (int wave = 0; wave < 4; ++wave)
      for (int lane = 0; lane < 64; ++lane) {
        const engram::dma::Lane l = engram::dma::lane_of(wave, lane, pitch);
        for (int i = 0; i < tile_rows / 32; ++i)
          for (int c = 0; c <= K / 256; ++c) {
            const uint32_t kofs = c < K / 256 ? (uint32_t)c * 128u : oob;
            const uint32_t v = engram::dma::voffset(l, i, kofs, pitch, oob, false);
            const int r = engram::dma::lds_row(wave, lane, i);
            expect(r < tile_rows, "LDS row past the chunk", r, tile_rows, i);
            const uint32_t piece = (uint32_t)((lane & 7) ^ engram::dma::swizzle(r));
            if (kofs != oob && r < rows)
              expect(v == (uint32_t)r * pitch + kofs + 16 * piece && (uint64_t)v + 16 <= range, "W piece", r, c, v);
            else
              expect((uint64_t)v >= range && v < 0x80000000u, "padding reads memory", r, c, v);
          }
      }
  }
}

}  // namespace

int main() {
  const int Ks[] = {128, 256, 384, 2048, 4096, 4224};
  for (int K : Ks)
    for (int rt : {1, 2, 5})
      for (int rows : {4, 12, 16, 20, 16 * rt})
        if (rows <= 16 * rt) gemv_w(rt, rows, K);
  for (int K : Ks)
    for (bool a8 : {false, true})
      for (int T : {1, 15, 16, 17, 33, 61, 64}) gemv_x(a8, (T + 15) / 16, T, K);
  for (uint32_t kb : {4u, 8u, 12u, 64u, 80u, 128u, 256u, 384u, 1024u, 1152u})
    for (int rt : {1, 2, 5})
      for (int rows : {4, 8, 16 * rt}) scales(rt, rows, kb);
  for (int tile : {256, 128})
    for (int total : {4, 100, 128, 132, 256, 300, 1284})
      for (int K : {256, 512, 2048}) gemm_w(total, K, tile);
  std::printf("fp4 dma model: %lld checks, %d failures\n", g_checks, g_fail);
  return g_fail == 0 ? 0 : 1;
}
