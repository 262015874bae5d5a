// The two microscaled 4-bit formats: E2M1 codes (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives), two to a byte (the element with the lower index in the
// low four bits), and one 8-bit scale per block of a row.
//   SQ_NVFP4: blocks of 16, scales E4M3, and one fp32 scale per row beside them
//   SQ_MXFP4: blocks of 32, scales E8M0 (a power of two, exponent + 127)
// Block scales are held in tiles of 128 rows x 4 blocks (512 bytes), the tiles
// of one row group back to back: the order in which the tensor cores' scale
// operand is copied to tensor memory (32 lanes of 16 bytes; lane l holds rows
// l, l + 32, l + 64 and l + 96).
#pragma once

#include <stdint.h>

namespace sq {

constexpr int kFp4TileRows = 128;
constexpr int kFp4TileBytes = 512;

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == 0 /* SQ_NVFP4 */ ? 16 : 32; }

// Scale tiles of one row group.
__host__ __device__ inline int64_t fp4_tiles_k(int fmt, int64_t K) {
    const int64_t blocks = (K + fp4_block(fmt) - 1) / fp4_block(fmt);
    return (blocks + 3) / 4;
}
__host__ __device__ inline int64_t fp4_tiles_m(int64_t rows) { return (rows + kFp4TileRows - 1) / kFp4TileRows; }

// Byte of the first of the four scales of `row` in tile column tk.
__device__ __forceinline__ int64_t fp4_scale_offset(int64_t row, int64_t tk, int64_t tiles_k) {
    const int r = (int)(row & 127);
    return ((row >> 7) * tiles_k + tk) * kFp4TileBytes + (r & 31) * 16 + (r >> 5) * 4;
}

}  // namespace sq
