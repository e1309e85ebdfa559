// Where a wave's loads stand in the packed weights of 4-bit experts, shared with the host.
#pragma once

#include "common.h"

namespace moe {

constexpr int kInt4Unit = 128;   // values of the contraction that are loaded together
constexpr int kInt4Blocks = 4;   // loads of a unit: a lane's four weight rows (gated: two gate rows, two up rows)

__host__ __device__ constexpr int64_t int4_row_bytes(int64_t K) { return 16 * ((K + 31) / 32); }

// The column whose weight row a wave's loads start from. A wave of a wide tile whose columns start behind the last takes
// those from 0 on, its results are not stored: behind the last the weights' resource would be empty, and a scalar
// offset that passes the end of a buffer resource leaves the range check nothing to compare with.
__host__ __device__ constexpr int64_t int4_first_column(int64_t n0, int64_t N) { return n0 < N ? n0 : 0; }

// Bytes from weight row r0 of an expert to the end of its last.
__host__ __device__ constexpr int64_t int4_bytes_left(int64_t w_rows, int64_t r0, int64_t row_bytes) {
  return r0 < w_rows ? (w_rows - r0) * row_bytes : 0;
}

// Scalar offset of load b of unit u: less than four weight rows, where there are at least eight.
__host__ __device__ constexpr uint32_t int4_block_at(bool gated, int b, int u, uint32_t row_bytes) {
  return (uint32_t)(gated ? b & 1 : b) * row_bytes + (uint32_t)u * (kInt4Unit / 2);
}

}  // namespace moe
