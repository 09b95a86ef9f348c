// Where the few-row kernels' loads point (ge_ffn_few.hip).  One set of functions for the device and
// for a CPU test that walks every lane of every load.
//
// A load reads 16 bytes at `offset` from a buffer that starts at the step's position and spans
// `extent` bytes; an offset at or past the extent reads zeros.  The range check covers the vector
// offset only -- a scalar offset is defined as excluded from it -- so the whole distance from the
// step's position is in the vector offset, and what lies past the last column or past K gets kFewOut.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ge {

constexpr uint32_t kFewOut = 0x80000000u;    // past every extent (leading dimensions are below 2^22 elements)

// `rows` rows of `left` values that remain of the contraction, row pitch ld2 bytes.
__host__ __device__ inline int few_row_extent(int rows, int left, uint32_t ld2) {
  return left > 0 ? (rows - 1) * (int)ld2 + left * 2 : 0;
}
// X: row l16, values 8 q16 + 32 half .. +7
__host__ __device__ inline uint32_t few_x_offset(uint32_t l16, uint32_t q16, int half, int left, uint32_t ldx2) {
  return (int)(8u * q16) + 32 * half < left ? l16 * ldx2 + 16u * q16 + 64u * (uint32_t)half : kFewOut;
}

// [N][K] weights, a row operand of `cols` rows: column 16 block + l16, values 8 q16 + 32 half .. +7
__host__ __device__ inline uint32_t few_nk_column(uint32_t l16, uint32_t q16, int block, int cols, uint32_t ldb2) {
  const uint32_t col = 16u * (uint32_t)block + l16;
  return (int)col < cols ? col * ldb2 + 16u * q16 : kFewOut;
}
__host__ __device__ inline uint32_t few_nk_offset(uint32_t column, uint32_t q16, int half, int left) {
  return (int)(8u * q16) + 32 * half < left ? column + 64u * (uint32_t)half : kFewOut;
}

// [K][N] weights, 32 values deep: value 8 q16 + k, columns 8 l16 .. +7
__host__ __device__ inline int few_kn_extent(int cols, int left, uint32_t ldb2) {
  return left > 0 ? ((left < 32 ? left : 32) - 1) * (int)ldb2 + cols * 2 : 0;
}
__host__ __device__ inline uint32_t few_kn_offset(uint32_t l16, uint32_t q16, int k, int cols, uint32_t ldb2) {
  return (int)(8u * l16) < cols ? (8u * q16 + (uint32_t)k) * ldb2 + 16u * l16 : kFewOut;
}

}  // namespace ge
