// dp_mx4.cuh -- the microscaled 4-bit formats, shared by their quantisation
// (dp_mx4.cu) and their product (dp_mx4mm.cu).
//
// A matrix [rows, cols] in 4 bits has e2m1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6
// and their negatives), two to a byte with the earlier column in the low half,
// rows cols / 2 bytes apart; and one 8-bit scale for each block of consecutive
// columns:
//   mxfp4  blocks of 32, a power of two (ue8m0: 2^(byte - 127), 255 is NaN)
//   nvfp4  blocks of 16, e4m3, times one fp32 scale of the whole tensor
// The scales lie as the tensor core takes them: tiles of 128 rows x 4 blocks,
// 512 bytes each, row r and block b of a tile at (r % 32) * 16 + (r / 32) * 4
// + b; the tiles of 128 rows follow one another along the columns.
#pragma once

#include "dp_common.cuh"

namespace dpk {

constexpr int kMxBlock = 32;  // mxfp4
constexpr int kNvBlock = 16;  // nvfp4
constexpr int kScaleTile = 512;
constexpr int kScaleRows = 128;

__host__ __device__ inline int mx4_block(dp_mx4_format_t f) {
  return f == DP_NVFP4 ? kNvBlock : kMxBlock;
}
// Scale tiles along the columns.
__host__ __device__ inline int mx4_col_tiles(int cols, int block) {
  return (cols + 4 * block - 1) / (4 * block);
}

}  // namespace dpk
