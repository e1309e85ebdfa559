// Grouped products of MXFP4 rows with MXFP4 expert weights, fp32 accumulation:
//
//   plain:  y[rows_e] = bf16( X_e W_e^T )                        W_e [N, K]
//   gated:  h[rows_e] = bf16( SiLU(g) * u ), [g | u] = X_e W_e^T   W_e [2N, K], gate rows first
//
// Every product of two 4-bit values and their blocks' powers of two is exact in fp32; sums are fp32,
// and there is one rounding, of the result (the gated form takes SiLU of the fp32 sums).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies 32 x 64 by 64 x 32: lane l brings one block of 32
// values (16 bytes) of row l % 32 and that block's scale byte. Which block of the row a lane brings
// is free as long as both operands agree, so lane half l / 32 takes neighbouring blocks: its values
// are contiguous and its scale bytes are one load. The weights are the first operand, so a lane ends
// with four consecutive columns of one row.

#include "mxfp4.h"

namespace moe {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

struct MxGemmArgs {
  const uint8_t* a_q;       // rows: [cap_rows, row bytes], or token rows [a_tokens, row bytes] when a_rows is set
  const uint8_t* a_s;
  const int32_t* a_rows;    // optional: sorted row p reads row a_rows[p] / a_k
  int a_k;
  int64_t a_tokens;
  const uint8_t* w_q;       // [E, w_rows, row bytes]
  const uint8_t* w_s;
  int64_t w_rows;           // weight rows per expert: N, gated 2N
  int64_t N, K;
  const int32_t* offsets;   // [E+1]
  int E;
  int64_t cap_rows;
  uint16_t* out;            // [cap_rows, N]
};

__device__ __forceinline__ i32x8 fp4_operand(const u32x4& v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// SiLU(g) * u in fp32 with the hardware exponential and reciprocal (a few fp32 ulps, far below the
// rounding of the result).
__device__ __forceinline__ float swiglu(float g, float u) { return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u; }

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t cap) { return v < 0 ? 0 : (v > cap ? cap : v); }

// ---------------------------------------------------------------------------------------------
// Few rows per expert: 32 rows by 64 weight rows a workgroup, operands straight from memory to
// registers, the contraction split over the four waves and joined through LDS.
// ---------------------------------------------------------------------------------------------
constexpr int kThinThreads = 256;
constexpr int kThinWaves = 4;
constexpr int kUnit = 128;  // contraction per step: four blocks, two per lane half

template <bool GATED>
__global__ __launch_bounds__(kThinThreads) void mxfp4_thin_kernel(MxGemmArgs g) {
  __shared__ int mt_prefix[MOE_MAX_EXPERTS + 1];
  __shared__ int wave_total[kThinWaves];
  __shared__ float4 red[kThinWaves * 2 * 4 * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 31, hh = lane >> 5;

  // prefix of the experts' 32-row tile counts, from the offsets clamped to the capacity
  {
    constexpr int kPer = MOE_MAX_EXPERTS / kThinThreads;
    int mt[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      mt[i] = 0;
      if (e < g.E) {
        const int64_t lo = clamp_row(g.offsets[e], g.cap_rows), hi = clamp_row(g.offsets[e + 1], g.cap_rows);
        mt[i] = hi > lo ? (int)((hi - lo + 31) / 32) : 0;
      }
      sum += mt[i];
    }
    int incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int up = __shfl_up(incl, off, 64);
      if (lane >= off) incl += up;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    int run = incl - sum;
    for (int w = 0; w < wave; ++w) run += wave_total[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= g.E) mt_prefix[e] = run;
      run += mt[i];
    }
    if (tid == kThinThreads - 1 && g.E == MOE_MAX_EXPERTS) mt_prefix[g.E] = run;
    __syncthreads();
  }
  constexpr int kCols = GATED ? 32 : 64;
  const int64_t n_tiles = (g.N + kCols - 1) / kCols;
  const int64_t total = (int64_t)mt_prefix[g.E] * n_tiles;
  const int64_t qp = mx_row_bytes(g.K), sp = mx_scale_bytes(g.K);
  const int blocks = (int)mx_blocks(g.K);
  const int units = (int)((g.K + kUnit - 1) / kUnit);
  const int u_lo = units * wave / kThinWaves, u_hi = units * (wave + 1) / kThinWaves;

  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int gm = (int)(t / n_tiles);
    const int64_t n0 = (t - (int64_t)gm * n_tiles) * kCols;
    int e = 0, hi_e = g.E;  // largest e with mt_prefix[e] <= gm
    while (hi_e - e > 1) {
      const int mid = (e + hi_e) >> 1;
      if (mt_prefix[mid] <= gm) e = mid; else hi_e = mid;
    }
    const int64_t lo = clamp_row(g.offsets[e], g.cap_rows), hi = clamp_row(g.offsets[e + 1], g.cap_rows);
    const int64_t row0 = lo + (int64_t)(gm - mt_prefix[e]) * 32;
    if (row0 < lo || row0 >= hi) continue;  // offsets that are no running sum can wrap the tile counts
    const int valid = (int)(hi - row0 < 32 ? hi - row0 : 32);
    // sources: rows past the block repeat its last, columns past N the tile's first; neither is stored
    int64_t a_row = row0 + (r < valid ? r : valid - 1);
    if (g.a_rows != nullptr) {
      const int64_t last = g.a_tokens * g.a_k - 1;
      int64_t slot = g.a_rows[a_row];
      slot = slot < 0 ? 0 : (slot > last ? last : slot);
      a_row = slot / g.a_k;
    }
    int64_t w_row[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      int64_t n = n0 + (GATED ? r : f * 32 + r);
      n = n < g.N ? n : n0;
      w_row[f] = e * g.w_rows + n + (GATED ? f * g.N : 0);
    }
    const uint8_t* a_q = g.a_q + a_row * qp;
    const uint8_t* a_s = g.a_s + a_row * sp;
    const uint8_t* w_q[2] = {g.w_q + w_row[0] * qp, g.w_q + w_row[1] * qp};
    const uint8_t* w_s[2] = {g.w_s + w_row[0] * sp, g.w_s + w_row[1] * sp};
    f32x16 acc[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
    for (int u = u_lo; u < u_hi; ++u) {
      const int b = 4 * u + 2 * hh;  // this half's blocks: b and b + 1
      u32x4 av[2], wv[2][2];
      uint32_t as, ws[2];
      const uint32_t keep = (b < blocks ? 0xFFu : 0u) | (b + 1 < blocks ? 0xFF00u : 0u);
      as = *reinterpret_cast<const uint16_t*>(a_s + b) & keep;
#pragma unroll
      for (int f = 0; f < 2; ++f) ws[f] = *reinterpret_cast<const uint16_t*>(w_s[f] + b) & keep;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const u32x4 zero{0u, 0u, 0u, 0u};
        const bool in = b + i < blocks;
        av[i] = in ? *reinterpret_cast<const u32x4*>(a_q + (b + i) * 16) : zero;
#pragma unroll
        for (int f = 0; f < 2; ++f) wv[f][i] = in ? *reinterpret_cast<const u32x4*>(w_q[f] + (b + i) * 16) : zero;
      }
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        acc[f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(wv[f][0]), fp4_operand(av[0]), acc[f], 4, 4, 0,
                                                                 (int)ws[f], 0, (int)as);
        acc[f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(wv[f][1]), fp4_operand(av[1]), acc[f], 4, 4, 1,
                                                                 (int)ws[f], 1, (int)as);
      }
    }
    // the waves' sums in wave order
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[((wave * 2 + f) * 4 + q) * 64 + lane] =
            float4{acc[f][4 * q], acc[f][4 * q + 1], acc[f][4 * q + 2], acc[f][4 * q + 3]};
    __syncthreads();
    float4 sum[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      sum[f] = red[(f * 4 + wave) * 64 + lane];  // this thread's quad of columns: q = wave
#pragma unroll
      for (int w = 1; w < kThinWaves; ++w) {
        const float4 v = red[((w * 2 + f) * 4 + wave) * 64 + lane];
        sum[f].x += v.x; sum[f].y += v.y; sum[f].z += v.z; sum[f].w += v.w;
      }
    }
    if (r < valid) {
      uint16_t* dst = g.out + (row0 + r) * g.N;
      const int64_t col = n0 + 8 * wave + 4 * hh;
      if constexpr (GATED) {
        if (col < g.N) {
          const uint2 v{pack_bf16x2(swiglu(sum[0].x, sum[1].x), swiglu(sum[0].y, sum[1].y)),
                        pack_bf16x2(swiglu(sum[0].z, sum[1].z), swiglu(sum[0].w, sum[1].w))};
          *reinterpret_cast<uint2*>(dst + col) = v;
        }
      } else {
#pragma unroll
        for (int f = 0; f < 2; ++f)
          if (col + 32 * f < g.N) {
            const uint2 v{pack_bf16x2(sum[f].x, sum[f].y), pack_bf16x2(sum[f].z, sum[f].w)};
            *reinterpret_cast<uint2*>(dst + col + 32 * f) = v;
          }
      }
    }
    __syncthreads();  // red is reused by the next tile
  }
}

template <bool GATED>
hipError_t launch_products(const MxGemmArgs& g, hipStream_t stream) {
  if (g.cap_rows == 0) return hipSuccess;
  const int cus = device_cu_count(current_device());
  hipLaunchKernelGGL(mxfp4_thin_kernel<GATED>, dim3(cus * 4), dim3(kThinThreads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_projection_mxfp4(const uint8_t* x_q, const uint8_t* x_s, const int32_t* offsets,
                                           const uint8_t* w_q, const uint8_t* w_s, int64_t cap_rows, int64_t d_in,
                                           int64_t d_out, int32_t E, uint16_t* y, hipStream_t stream) {
  const MxGemmArgs g{x_q, x_s, nullptr, 1, 0, w_q, w_s, d_out, d_out, d_in, offsets, E, cap_rows, y};
  return launch_products<false>(g, stream);
}

hipError_t launch_gemm_up_swiglu_mxfp4(const uint8_t* x_q, const uint8_t* x_s, int64_t x_rows, const int32_t* perm,
                                       int32_t k, const int32_t* offsets, const uint8_t* w_q, const uint8_t* w_s,
                                       int64_t cap_rows, int64_t d, int64_t h, int32_t E, uint16_t* h_buf,
                                       hipStream_t stream) {
  const MxGemmArgs g{x_q, x_s, perm, k, x_rows, w_q, w_s, 2 * h, h, d, offsets, E, cap_rows, h_buf};
  return launch_products<true>(g, stream);
}

}  // namespace moe
