// mx.cuh -- the layout of microscaled 4-bit matrices (include/zipnn.h) on host and device.
#pragma once
#include <cstdint>

#include "zipnn.h"

namespace zipnn {

constexpr int kMxFp4 = 0, kNvFp4 = 1;
constexpr int kValBF16 = 0, kValFP32 = 1, kValFP16 = 2;
constexpr uint32_t kMxTileBytes = 512;  // scales of 128 rows x 4 blocks

__host__ __device__ constexpr uint32_t mx_block(int fmt) { return fmt == kMxFp4 ? 32u : 16u; }
__host__ __device__ constexpr uint64_t mx_div_up(uint64_t a, uint64_t b) { return a / b + (a % b != 0); }
__host__ __device__ constexpr uint64_t mx_row_bytes(uint64_t cols) { return 16 * mx_div_up(cols, 32); }
// tiles along a row
__host__ __device__ constexpr uint64_t mx_col_tiles(int fmt, uint64_t cols) { return mx_div_up(cols, 4ull * mx_block(fmt)); }
// byte of (row, block) in the tile that holds it
__host__ __device__ constexpr uint32_t mx_in_tile(uint32_t row, uint32_t block) {
  return 16 * (row % 32) + 4 * (row / 32 % 4) + block % 4;
}
// The largest sizes a call takes: every byte offset stays far inside 64 bits, and a place in a
// row inside an int.
constexpr uint64_t kMxMaxRows = 1ull << 31, kMxMaxCols = 1ull << 30, kMxMaxStride = 1ull << 40;
inline bool mx_valid(int fmt, uint64_t rows, uint64_t cols) {
  return (fmt == kMxFp4 || fmt == kNvFp4) && rows >= 1 && cols >= 1 && rows <= kMxMaxRows && cols <= kMxMaxCols;
}
// Matrices whose largest value every block of a quantisation finds for itself.
inline bool mx_small(uint64_t rows, uint64_t cols) { return rows <= ZIPNN_MX_SMALL && rows * mx_div_up(cols, 32) <= ZIPNN_MX_SMALL; }
inline bool mx_valid_type(int t) { return t == kValBF16 || t == kValFP32 || t == kValFP16; }
__host__ __device__ constexpr uint32_t mx_value_bytes(int t) { return t == kValFP32 ? 4u : 2u; }

}  // namespace zipnn
