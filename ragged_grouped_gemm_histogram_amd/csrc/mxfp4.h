// Sizes and per-lane conversions of MXFP4 rows, shared by the quantising kernels and the products.
#pragma once

#include "common.h"

namespace moe {

__host__ __device__ __forceinline__ int64_t mx_blocks(int64_t K) { return (K + 31) / 32; }
__host__ __device__ __forceinline__ int64_t mx_row_bytes(int64_t K) { return 16 * mx_blocks(K); }
__host__ __device__ __forceinline__ int64_t mx_scale_bytes(int64_t K) { return 16 * ((K + 511) / 512); }

// Where stage `stage` of a packed row (kMxStageBlocks blocks) starts, in bytes. Stages past the row's last take that
// one's start: a scalar offset that passes the end of a buffer resource leaves the range check nothing to compare with.
constexpr int kMxStageBlocks = 4;
__host__ __device__ constexpr uint32_t mx_stage_offset(int stage, int blocks) {
  const int last = (blocks - 1) / kMxStageBlocks;
  return (uint32_t)(stage < last ? stage : last) * (16u * kMxStageBlocks);
}

// Tiles of `height` rows that the rows [lo, hi) take, 0 <= lo; none if hi is before lo. In unsigned arithmetic: a block
// may have 2^31 - 1 rows.
__host__ __device__ constexpr uint32_t mx_row_tiles(int lo, int hi, int height) {
  return hi > lo ? ((uint32_t)hi - (uint32_t)lo + (uint32_t)height - 1u) / (uint32_t)height : 0u;
}

typedef __bf16 mx_bf16x2 __attribute__((ext_vector_type(2)));

template <int CTRL>
__device__ __forceinline__ uint32_t quad_xor(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}

// Largest bf16 magnitude (as bits: they order like the values, infinities and NaNs on top) of 8 values.
__device__ __forceinline__ uint32_t max_magnitude(const u32x4& v) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
  return m;
}

// The block's scale byte from its largest magnitude: the exponent field (the value's own exponent
// + 127) less 2, at least 0; 255 where the largest is not finite.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  const uint32_t field = top >> 7;
  return field == 255u ? 255u : (field > 2u ? field - 2u : 0u);
}

// 8 bf16 values to 8 4-bit floats at a block's scale (value 0 lowest). The convert takes the scale
// as the fp32 number 2^e, whose exponent field is the scale byte itself; a block that is not finite
// gets zeros.
__device__ __forceinline__ mx_bf16x2 bf16_pair(uint32_t bits) { return __builtin_bit_cast(mx_bf16x2, bits); }

__device__ __forceinline__ uint32_t to_fp4(const u32x4& v, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16_pair(v[0]), scale, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16_pair(v[1]), scale, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16_pair(v[2]), scale, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, bf16_pair(v[3]), scale, 3);
  return byte == 255u ? 0u : r;
}

__device__ __forceinline__ u32x4 from_fp4(uint32_t code, uint32_t byte) {
  const float scale = __uint_as_float(byte << 23);
  u32x4 v;
  v[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 0));
  v[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 1));
  v[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 2));
  v[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(code, scale, 3));
  if (byte == 255u) v = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
  return v;
}

}  // namespace moe
