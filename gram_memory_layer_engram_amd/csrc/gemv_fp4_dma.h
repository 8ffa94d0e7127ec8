// Offsets of the MXFP4 GEMV's global -> LDS DMAs and of the LDS reads that
// follow them (gemv_mxfp4.hip), in a form the host can evaluate too:
// tests/fp4_dma_model.cpp walks them on the CPU.
//
// A DMA writes LDS at base + lane * 16. A raw buffer load range-checks its
// vector offset alone: a lane's vector offset is its row and its piece inside
// the step, the step's offset inside the row rides in the unchecked scalar
// offset. With num_records = rows * pitch a lane whose row exists reads inside
// its row (the scalar offset is a whole number of steps of that row), and a
// lane whose row does not exist is past the range whatever the step.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace engram {
namespace fp4 {

// W: 64 bytes a row and step (128 k), 16 rows a DMA; piece p (of 4) of row r
// at p ^ ((r >> 1) & 3).
constexpr int kWStep = 64;
__host__ __device__ inline uint32_t w_voffset(int lane, int rt, int pitch) {
  return (uint32_t)((rt * 16 + (lane >> 2)) * pitch + (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
}
// the 16 bytes of k 32g .. 32g+31 of row r (0..15) in a row tile's 1 KiB
__host__ __device__ inline int w_read(int r, int g) { return r * 64 + ((g ^ ((r >> 1) & 3)) << 4); }

// x: 256 bytes a row and step in bf16 (4 rows a DMA), 128 in MXFP8 (8 rows);
// piece p of row r at p ^ (r & 7).
__host__ __device__ constexpr int x_step(bool a8) { return a8 ? 128 : 256; }
__host__ __device__ inline uint32_t x_voffset(bool a8, int lane, int token0, int i, int pitch) {
  const int rows = a8 ? 8 : 4, pieces = 64 / rows;
  const int row = i * rows + lane / pieces;
  return (uint32_t)((token0 + row) * pitch + (((lane % pieces) ^ (row & 7)) << 4));
}
// piece p of token r (0..15) in a token tile
__host__ __device__ inline int x_read(bool a8, int r, int p) { return r * x_step(a8) + ((p ^ (r & 7)) << 4); }

// Scale bytes of a workgroup's rows, kb a row, contiguous; `swap` (kb % 128 ==
// 0) exchanges the 16-byte pieces of a row by its number: the row's XOR on
// byte offsets, the global byte that belongs at LDS byte ofs (a multiple of
// 16), and the LDS byte of byte b of a row.
__host__ __device__ inline uint32_t s_xor(bool swap, uint32_t row, uint32_t kb) {
  return swap ? (kb % 256 == 0 ? row & 15u : (row & 15u) >> 1) << 4 : 0u;
}
__host__ __device__ inline uint32_t s_source(bool swap, uint32_t ofs, uint32_t kb) {
  const uint32_t row = swap ? ofs / kb : 0u;
  return row * kb + ((ofs - row * kb) ^ s_xor(swap, row, kb));
}
__host__ __device__ inline uint32_t s_read(bool swap, uint32_t row, uint32_t b, uint32_t kb) {
  return row * kb + (b ^ s_xor(swap, row, kb));
}

}  // namespace fp4
}  // namespace engram
