// Offsets of the int8 GEMV's global -> LDS DMAs and of the LDS reads that follow
// them (gemv_int8.hip), in a form the host can evaluate too:
// tests/int8_dma_model.cpp walks them on the CPU.
//
// A step is 128 k of 16 rows: 2 KiB, two DMAs of 8 rows x 128 bytes (8 whole
// cache lines). Lane l of DMA i writes LDS row 8i + l/8, position l%8, and
// fetches the row's piece (l%8) ^ (row & 7), so that the rows a fragment read
// touches lie on distinct banks.
//
// A raw buffer load range-checks its vector offset alone, so the whole offset
// (row, step, piece) travels in it: with num_records = rows * K a piece past the
// last row reads zeros, and so does a step that does not exist (kofs = kOob). A
// piece past its row's end (K % 128 != 0) reads the next row's bytes or zeros: of
// the two factors of a product one has to be zeros there, which is x.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace engram {
namespace i8 {

constexpr int kStep = 128;             // k, and bytes of a row
constexpr int kTileBytes = 16 * kStep;
constexpr uint32_t kOob = 0x70000000u;  // past every range, with a row's offset (at most 2^28) added still below 2^31

// byte offset inside its row's step of the piece that lane l fetches (the same for every DMA)
__host__ __device__ inline uint32_t piece_of(int lane) { return (uint32_t)(((lane & 7) ^ ((lane >> 3) & 7)) << 4); }
// vector offset of DMA q (rows 8q .. 8q+7) for the step at byte kofs of the rows, or kOob
__host__ __device__ inline uint32_t voffset(int lane, int q, uint32_t kofs, uint32_t K) {
  return (uint32_t)(q * 8 + (lane >> 3)) * K + piece_of(lane) + kofs;
}
// piece p (0..7) of row r (0..15) in a tile's 2 KiB
__host__ __device__ inline int read(int r, int p) { return r * kStep + ((p ^ (r & 7)) << 4); }

}  // namespace i8
}  // namespace engram
