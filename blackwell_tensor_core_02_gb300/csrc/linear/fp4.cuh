// fp4.cuh -- the layout of a microscaled 4-bit matrix (see linear_ops.h), for
// host and device.
#pragma once

#include <stdint.h>

namespace linear_ops {

constexpr int kScaleTileRows = 128;   // rows of a scale tile
constexpr int kScaleTileBytes = 512;  // 128 rows x 4 blocks

__host__ __device__ constexpr int fp4_block(bool nv) { return nv ? 16 : 32; }

// Columns as stored: whole 16-byte units of data.
__host__ __device__ constexpr int64_t fp4_padded_cols(int64_t cols) { return (cols + 31) / 32 * 32; }

// Scale tiles along the columns.
__host__ __device__ constexpr int64_t fp4_scale_tiles(int64_t cols, bool nv) {
    return (fp4_padded_cols(cols) / fp4_block(nv) + 3) / 4;
}

// Byte of the scale of (row, block), tiles = fp4_scale_tiles().
__host__ __device__ constexpr int64_t fp4_scale_at(int64_t row, int64_t block, int64_t tiles) {
    return ((row / kScaleTileRows) * tiles + block / 4) * kScaleTileBytes + (row % 32) * 16 + (row % 128) / 32 * 4 +
           block % 4;
}

}  // namespace linear_ops
