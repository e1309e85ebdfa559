// MXFP4 (OCP Microscaling Formats v1.0, MXFP4): blocks of 32 values share a power of two, kept as the
// byte e + 127 (255 marks a block that held an infinity or a NaN); each value is a 4-bit float E2M1
// (magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6). A block's exponent is e = floor(log2 max|x|) - 2, not below
// -127; values are rounded to nearest even and saturate at 6. A packed row of K values is
// 16 * ceil(K / 32) bytes (value 2i in the low half of byte i) and its scale bytes are
// 16 * ceil(K / 512), zeros behind the last block.
//
// Quantising and reading back are one pass over memory: 2 bytes in and 17/32 out per value (the
// other way round back), so both are bound by HBM. A quad of lanes holds one block, 8 values (16
// bytes) a lane; the block's maximum takes two lane exchanges and the conversion four packed
// convert instructions a lane.

#include "mxfp4.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Pieces of 8 values a thread has in flight. The bf16 side is streamed (non-temporal: it is read or
// written once, and passes the caches by). Measured on 65536 x 2048, 340 MB either way: quantising 2
// pieces 61 to 65 us (1: 61, 4: 65; with ordinary loads 63 to 66), reading back 2 pieces 48.5 us
// (4: 50, 8: 51; with ordinary stores 62). At 4096 x 2048, between kernels that write the input and
// read the output, streaming costs nothing (15.0 and 15.1 us for the pair, 15.3 and 15.7 without).
constexpr int kQuantizeChunks = 2, kDequantizeChunks = 2;

// Rows of K-contiguous values. Work item: 8 consecutive values of a row padded to whole blocks; a
// workgroup takes kThreads * kQuantizeChunks consecutive items.
__global__ __launch_bounds__(kThreads) void mxfp4_quantize_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t K,
                                                                  uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
  const int64_t cpr = mx_blocks(K) * 4;  // items per row
  const int64_t total = rows * cpr;
  const int64_t span = (int64_t)kThreads * kQuantizeChunks;
  const int64_t first = (int64_t)blockIdx.x * span;
  const int64_t row0 = first / cpr;
  const int rem0 = (int)(first - row0 * cpr);
  const float inv = 1.0f / (float)cpr;
  u32x4 v[kQuantizeChunks];
  int64_t row[kQuantizeChunks];
  int chunk[kQuantizeChunks];
#pragma unroll
  for (int i = 0; i < kQuantizeChunks; ++i) {
    // rem0 + local < 2^24: the fp32 quotient is off by at most one
    const int local = rem0 + i * kThreads + (int)threadIdx.x;
    int r = (int)((float)local * inv);
    int c = local - r * (int)cpr;
    if (c < 0) { --r; c += (int)cpr; }
    if (c >= cpr) { ++r; c -= (int)cpr; }
    row[i] = row0 + r;
    chunk[i] = c;
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (row[i] < rows && (int64_t)c * 8 < K) v[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + row[i] * K + (int64_t)c * 8));
  }
  const int64_t qp = mx_row_bytes(K), sp = mx_scale_bytes(K);
#pragma unroll
  for (int i = 0; i < kQuantizeChunks; ++i) {
    if (first + i * kThreads + threadIdx.x >= total) continue;  // whole quads: total is a multiple of 4
    uint32_t top = max_magnitude(v[i]);
    top = max(top, quad_xor<0xB1>(top));
    top = max(top, quad_xor<0x4E>(top));
    const uint32_t byte = scale_byte(top);
    reinterpret_cast<uint32_t*>(q + row[i] * qp)[chunk[i]] = to_fp4(v[i], byte);
    if ((chunk[i] & 3) == 0) {
      const int64_t b = chunk[i] >> 2;
      uint8_t* s = scales + row[i] * sp;
      s[b] = (uint8_t)byte;
      if (b == mx_blocks(K) - 1)
        for (int64_t z = b + 1; z < sp; ++z) s[z] = 0;
    }
  }
}

// Weights stored with the contraction outermost, [E, K, N]: the packed rows are the columns. A
// workgroup turns 128 columns of 16 blocks (512 k): a lane takes two neighbouring columns of one
// block at a time (4-byte loads, 256 contiguous bytes a wave), and the packed rows leave through LDS,
// 256 bytes of values and 16 of scales each. 16 x 2880 x 2880 (336 MB) take 65 us, 5.2 TB/s: with
// ordinary loads 81, with four columns a lane (8-byte loads, half the blocks) 68; with the rows
// written from the lanes that made them, 16 bytes and one byte a row, 114, the single bytes 20 of them.
constexpr int kTileCols = 128, kTileBlocks = 16, kRowPitch = kTileBlocks * 16 + 16;

__global__ __launch_bounds__(kThreads) void mxfp4_quantize_columns_kernel(const uint16_t* __restrict__ x, int64_t K, int64_t N,
                                                                          uint8_t* __restrict__ q,
                                                                          uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t rows[kTileCols * kRowPitch];
  __shared__ __align__(16) uint8_t bytes[kTileCols * kTileBlocks];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * kTileCols, b0 = (int64_t)blockIdx.y * kTileBlocks, e = blockIdx.z;
  const int64_t n = n0 + 2 * lane, blocks = mx_blocks(K);
#pragma unroll 1
  for (int bi = wave; bi < kTileBlocks; bi += kThreads / 64) {
    const int64_t k0 = (b0 + bi) * 32;
    uint32_t v[32];
    const uint16_t* src = x + (e * K + k0) * N + n;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      v[i] = n < N && k0 + i < K ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(src + (int64_t)i * N)) : 0u;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      u32x4 part[4], out;
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t a = v[8 * c + 2 * w], d = v[8 * c + 2 * w + 1];
          part[c][w] = half == 0 ? (a & 0xFFFFu) | (d << 16) : (a >> 16) | (d & 0xFFFF0000u);
        }
        top = max(top, max_magnitude(part[c]));
      }
      const uint32_t byte = scale_byte(top);
#pragma unroll
      for (int c = 0; c < 4; ++c) out[c] = to_fp4(part[c], byte);
      *reinterpret_cast<u32x4*>(rows + (2 * lane + half) * kRowPitch + bi * 16) = out;
      bytes[(2 * lane + half) * kTileBlocks + bi] = (uint8_t)byte;  // 0 past the row's last block
    }
  }
  __syncthreads();
  const int64_t qp = mx_row_bytes(K), sp = mx_scale_bytes(K);
#pragma unroll
  for (int i = tid; i < kTileCols * kTileBlocks; i += kThreads) {
    const int r = i / kTileBlocks, c = i % kTileBlocks;
    if (n0 + r < N && b0 + c < blocks)
      *reinterpret_cast<u32x4*>(q + (e * N + n0 + r) * qp + (b0 + c) * 16) =
          *reinterpret_cast<const u32x4*>(rows + r * kRowPitch + c * 16);
  }
  if (tid < kTileCols && n0 + tid < N)
    *reinterpret_cast<u32x4*>(scales + (e * N + n0 + tid) * sp + b0) =
        *reinterpret_cast<const u32x4*>(bytes + tid * kTileBlocks);
}

// Packed rows back to bf16: a 4-bit value times a power of two has two significant bits and at least
// 2^-128, which bf16's smallest normals and subnormals hold, and at most 6 * 2^(byte - 127), which
// bf16 holds up to byte 252. Rows quantised here have at most that; beyond, values that bf16 does not
// hold become infinities.
__global__ __launch_bounds__(kThreads) void mxfp4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                    const uint8_t* __restrict__ scales, int64_t rows,
                                                                    int64_t K, uint16_t* __restrict__ x) {
  const int64_t cpr = K / 8;
  const int64_t span = (int64_t)kThreads * kDequantizeChunks;
  const int64_t first = (int64_t)blockIdx.x * span;
  const int64_t row0 = first / cpr;
  const int rem0 = (int)(first - row0 * cpr);
  const float inv = 1.0f / (float)cpr;
  const int64_t qp = mx_row_bytes(K), sp = mx_scale_bytes(K);
  uint32_t code[kDequantizeChunks], byte[kDequantizeChunks];
  int64_t at[kDequantizeChunks];
#pragma unroll
  for (int i = 0; i < kDequantizeChunks; ++i) {
    const int local = rem0 + i * kThreads + (int)threadIdx.x;
    int r = (int)((float)local * inv);
    int c = local - r * (int)cpr;
    if (c < 0) { --r; c += (int)cpr; }
    if (c >= cpr) { ++r; c -= (int)cpr; }
    const int64_t row = row0 + r;
    at[i] = row < rows ? row * K + (int64_t)c * 8 : -1;
    if (row < rows) {
      code[i] = reinterpret_cast<const uint32_t*>(q + row * qp)[c];
      byte[i] = scales[row * sp + (c >> 2)];
    }
  }
#pragma unroll
  for (int i = 0; i < kDequantizeChunks; ++i)
    if (at[i] >= 0) __builtin_nontemporal_store(from_fp4(code[i], byte[i]), reinterpret_cast<u32x4*>(x + at[i]));
}

}  // namespace

namespace {

// A launch has at most 2^32 - 1 work items; rows of more pieces (2^36 values and up) take several.
template <typename F>
hipError_t by_rows(int64_t rows, int64_t items_per_row, int chunks, F&& launch) {
  const int64_t span = (int64_t)kThreads * chunks;
  const int64_t most = ((int64_t(1) << 32) / kThreads - 1) * span / items_per_row;  // K <= 2^24: at least 2^10 rows
  for (int64_t r0 = 0; r0 < rows; r0 += most) {
    const int64_t n = rows - r0 < most ? rows - r0 : most;
    launch(r0, n, dim3((unsigned)((n * items_per_row + span - 1) / span)));
    const hipError_t st = hipGetLastError();
    if (st != hipSuccess) return st;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_mxfp4_quantize(const uint16_t* x, int64_t rows, int64_t K, uint8_t* q, uint8_t* scales,
                                 hipStream_t stream) {
  return by_rows(rows, mx_blocks(K) * 4, kQuantizeChunks, [&](int64_t r0, int64_t n, dim3 grid) {
    hipLaunchKernelGGL(mxfp4_quantize_kernel, grid, dim3(kThreads), 0, stream, x + r0 * K, n, K, q + r0 * mx_row_bytes(K),
                       scales + r0 * mx_scale_bytes(K));
  });
}

hipError_t launch_mxfp4_quantize_columns(const uint16_t* x, int64_t K, int64_t N, int32_t E, uint8_t* q,
                                         uint8_t* scales, hipStream_t stream) {
  const dim3 grid((unsigned)((N + kTileCols - 1) / kTileCols), (unsigned)((mx_blocks(K) + kTileBlocks - 1) / kTileBlocks),
                  (unsigned)E);
  hipLaunchKernelGGL(mxfp4_quantize_columns_kernel, grid, dim3(kThreads), 0, stream, x, K, N, q, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* q, const uint8_t* scales, int64_t rows, int64_t K, uint16_t* x,
                                   hipStream_t stream) {
  return by_rows(rows, K / 8, kDequantizeChunks, [&](int64_t r0, int64_t n, dim3 grid) {
    hipLaunchKernelGGL(mxfp4_dequantize_kernel, grid, dim3(kThreads), 0, stream, q + r0 * mx_row_bytes(K),
                       scales + r0 * mx_scale_bytes(K), n, K, x + r0 * K);
  });
}

}  // namespace moe
