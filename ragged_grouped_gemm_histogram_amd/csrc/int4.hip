// Expert weights in 4 bits with a scale per group of values along the contraction, W = s (q - z), and the
// grouped products of bf16 rows with them, fp32 accumulation, one rounding of the result:
//
//   plain:  y[rows_e] = bf16( X_e W_e^T )                          W_e [N, K]
//   gated:  h[rows_e] = bf16( SiLU(g) * u ), [g | u] = X_e W_e^T   W_e [2N, K], gate rows first
//
// For decode: few rows an expert, bound by reading the weights of the experts that have rows. A packed
// weight becomes a bf16 by putting its four bits into the mantissa of 16: 16 + q is exact, two weights
// take a shift and one and-or. The matrix instruction then gives A = sum (16 + q) x over a group, one more
// with ones for weights gives B = sum x, and the group adds s (A - (16 + z) B) to the result.
//
// v_mfma_f32_16x16x32_bf16: lane l brings 8 values of row l % 16, those of lane quarter l / 16. A
// lane loads 16 bytes, 32 weights of one row; exchanging dwords between the four quarters makes step s of
// four cover values 32 s .. 32 s + 31 of a unit of 128, so that groups of 32, 64 and 128 all end with
// a step. The weights are the first operand, so a lane ends with four consecutive columns of one token.

#include <type_traits>

#include "grouped.h"

namespace moe {
namespace {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct Int4Args {
  const uint16_t* x;        // rows [cap_rows, K], or token rows read through perm
  const int32_t* perm;      // optional: sorted row p reads row perm[p] / k
  int k;
  int64_t tokens;
  const uint8_t* q;         // [E, w_rows, row bytes]
  const uint16_t* scales;   // [E, groups, w_rows]
  const uint8_t* zeros;     // the same shape, or NULL: 8
  int group;                // 32, 64 or 128
  int64_t w_rows, N, K;     // weight rows an expert: N, gated 2N
  const int32_t* offsets;
  int E;
  int64_t cap_rows;
  uint16_t* out;            // [cap_rows, N]
};

inline __host__ __device__ int64_t int4_row_bytes(int64_t K) { return 16 * ((K + 31) / 32); }

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __builtin_bit_cast(float, x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __builtin_bit_cast(float, x & 0xFFFF0000u); }

// Eight weights of a dword as bf16 16 + q, in the order 0 4, 1 5, 2 6, 3 7.
__device__ __forceinline__ bf16x8 unpack(uint32_t w) {
  constexpr uint32_t kBits = 0x00780078u, kSixteen = 0x41804180u;
  const u32x4 v = {((w << 3) & kBits) | kSixteen, ((w >> 1) & kBits) | kSixteen, ((w >> 5) & kBits) | kSixteen,
                   ((w >> 9) & kBits) | kSixteen};
  return __builtin_bit_cast(bf16x8, v);
}

// Eight bf16 of a row in the weights' order.
__device__ __forceinline__ bf16x8 pair_up(u32x4 x) {
  const u32x4 v = {__builtin_amdgcn_perm(x[2], x[0], 0x05040100u), __builtin_amdgcn_perm(x[2], x[0], 0x07060302u),
                   __builtin_amdgcn_perm(x[3], x[1], 0x05040100u), __builtin_amdgcn_perm(x[3], x[1], 0x07060302u)};
  return __builtin_bit_cast(bf16x8, v);
}

// Dword d of lane quarter g becomes dword g of lane quarter d.
__device__ __forceinline__ void transpose_quarters(u32x4& w) {
  const auto a = __builtin_amdgcn_permlane32_swap(w[0], w[2], false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(w[1], w[3], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w = u32x4{c[0], c[1], d[0], d[1]};
}

constexpr int kThreads = 256;
constexpr int kWaves = 4;
constexpr int kUnit = 128;
constexpr int kBlocks = 4;  // blocks of 16 weight rows of a tile

// Row tiles of an expert.
__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t cap) { return v < 0 ? 0 : (v > cap ? cap : v); }

// A tile: 16 MB rows by 64 weight rows (gated: 32 columns' gate and up rows), the contraction dealt to the
// four waves in units of 128 and joined through LDS.
template <bool GATED, int MB>
__global__ __launch_bounds__(kThreads, MB == 1 ? 4 : 2) void int4_kernel(Int4Args g) {
  constexpr int BM = 16 * MB, kCols = GATED ? 32 : 64;
  __shared__ int prefix[MOE_MAX_EXPERTS + 1];
  __shared__ int offs[MOE_MAX_EXPERTS + 1];
  __shared__ uint32_t wave_total[kWaves];
  __shared__ f32x4_t red[kWaves * kBlocks * MB * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int quarter = lane >> 4, r16 = lane & 15;

  // prefix of the experts' row tiles
  {
    constexpr int kPer = MOE_MAX_EXPERTS / kThreads;
    uint32_t mt[kPer], sum = 0;  // (unsigned: offsets that are no running sum can wrap the counts)
    for (int e = tid; e <= g.E; e += kThreads) offs[e] = (int)clamp_row(g.offsets[e], g.cap_rows);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      const int rows = e < g.E ? offs[e + 1] - offs[e] : 0;
      mt[i] = rows > 0 ? (uint32_t)(rows + BM - 1) / BM : 0u;
      sum += mt[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t up = __shfl_up(incl, off, 64);
      if (lane >= off) incl += up;
    }
    if (lane == 63) wave_total[wave] = incl;
    __syncthreads();
    uint32_t run = incl - sum;
    for (int w = 0; w < wave; ++w) run += wave_total[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= g.E) prefix[e] = (int)run;
      run += mt[i];
    }
    if (tid == kThreads - 1 && g.E == MOE_MAX_EXPERTS) prefix[g.E] = (int)run;
    __syncthreads();
  }
  const int n_tiles = (int)((g.N + kCols - 1) / kCols);
  const int64_t total = (int64_t)prefix[g.E] * n_tiles;
  const int64_t row_bytes = int4_row_bytes(g.K);
  const int units = (int)((g.K + kUnit - 1) / kUnit);
  const int groups = (int)((g.K + g.group - 1) / g.group);
  const int steps = g.group / 32;  // matrix steps of a group
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const int gm = (int)(tile / n_tiles);
    const int n0 = (int)(tile - (int64_t)gm * n_tiles) * kCols;
    int e = 0, hi_e = g.E;  // largest e with prefix[e] <= gm
    while (hi_e - e > 1) {
      const int mid = (e + hi_e) >> 1;
      if (prefix[mid] <= gm) e = mid; else hi_e = mid;
    }
    const int64_t lo = offs[e], hi = offs[e + 1];
    const int64_t row0 = lo + ((int64_t)gm - prefix[e]) * BM;
    if (row0 < lo || row0 >= hi) continue;  // wrapped counts
    const int valid = (int)(hi - row0 < BM ? hi - row0 : BM);

    // sources: weight rows past the last repeat it, they are not stored
    const uint16_t* xr[MB];
    bool has[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int t = m * 16 + r16;
      has[m] = t < valid;
      int64_t row = row0 + (has[m] ? t : 0);
      if (g.perm != nullptr) row = clamp_row((int64_t)g.perm[row] / g.k, g.tokens - 1);
      xr[m] = g.x + row * g.K;
    }
    const uint8_t* wr[kBlocks];
    int64_t sr[kBlocks];  // this lane's four columns' scales, first group
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const int part = GATED ? b >> 1 : 0;                       // gate or up
      const int64_t c0 = n0 + (GATED ? b & 1 : b) * 16;
      int64_t row = c0 + r16, col = c0 + quarter * 4;
      row = (row < g.N ? row : g.N - 1) + part * g.N;
      col = (col < g.N ? col : g.N - 4) + part * g.N;
      wr[b] = g.q + ((int64_t)e * g.w_rows + row) * row_bytes;
      sr[b] = (int64_t)e * groups * g.w_rows + col;
    }

    f32x4_t sum[kBlocks][MB];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) sum[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    for (int u = wave; u < units; u += kWaves) {
      u32x4 w[kBlocks], x[MB][4];
      const int64_t wb = (int64_t)u * 64 + quarter * 16;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        w[b] = u32x4{0u, 0u, 0u, 0u};
        if (wb < row_bytes) w[b] = *reinterpret_cast<const u32x4*>(wr[b] + wb);
      }
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t kk = (int64_t)u * kUnit + s * 32 + quarter * 8;
          x[m][s] = u32x4{0u, 0u, 0u, 0u};
          if (has[m] && kk < g.K) x[m][s] = *reinterpret_cast<const u32x4*>(xr[m] + kk);
        }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) transpose_quarters(w[b]);
      f32x4_t acc[kBlocks][MB], xs[MB];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const bool first = (s & (steps - 1)) == 0, last = (s & (steps - 1)) == steps - 1;
        bf16x8 xv[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[m] = pair_up(x[m][s]);
        if (first) {
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            xs[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) acc[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, xv[m], xs[m], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const bf16x8 wv = unpack(w[b][s]);
#pragma unroll
          for (int m = 0; m < MB; ++m) acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wv, xv[m], acc[b][m], 0, 0, 0);
        }
        if (last) {
          int gi = (u * 4 + s) / steps;
          gi = gi < groups ? gi : groups - 1;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const int64_t at = sr[b] + (int64_t)gi * g.w_rows;
            const u32x2_t sc = *reinterpret_cast<const u32x2_t*>(g.scales + at);
            const uint32_t z = g.zeros != nullptr ? *reinterpret_cast<const uint32_t*>(g.zeros + at) : 0x08080808u;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float scale = r & 1 ? bf16_hi(sc[r >> 1]) : bf16_lo(sc[r >> 1]);
              const float c = 16.0f + (float)((z >> (8 * r)) & 0xFFu);
#pragma unroll
              for (int m = 0; m < MB; ++m) sum[b][m][r] = fmaf(scale, fmaf(-c, xs[m][r], acc[b][m][r]), sum[b][m][r]);
            }
          }
        }
      }
    }
    // join the waves' parts
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) red[((wave * kBlocks + b) * MB + m) * 64 + lane] = sum[b][m];
    __syncthreads();
    constexpr int kItems = (GATED ? 2 : 4) * MB;  // blocks of 16 tokens by 16 columns
    for (int i = wave; i < kItems; i += kWaves) {
      const int b = i / MB, m = i % MB;
      f32x4_t v = red[(b * MB + m) * 64 + lane];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += red[((w * kBlocks + b) * MB + m) * 64 + lane];
      if constexpr (GATED) {
        f32x4_t up = red[((b + 2) * MB + m) * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) up += red[((w * kBlocks + b + 2) * MB + m) * 64 + lane];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = v[r] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[r])) * up[r];
      }
      const int t = m * 16 + r16;
      const int64_t col = n0 + b * 16 + quarter * 4;
      if (t < valid && col < g.N)
        *reinterpret_cast<u32x2_t*>(g.out + (row0 + t) * g.N + col) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
    __syncthreads();
  }
}

template <bool GATED, int MB>
hipError_t launch_tiles(const Int4Args& g, hipStream_t stream) {
  constexpr int BM = 16 * MB;
  const int64_t n_tiles = (g.N + (GATED ? 31 : 63)) / (GATED ? 32 : 64);
  const int64_t most_experts = g.cap_rows < g.E ? g.cap_rows : g.E;
  const int64_t tiles = (g.cap_rows / BM + most_experts) * n_tiles;
  const int64_t fit = (int64_t)device_cu_count(current_device()) * (MB == 1 ? 4 : 2);
  hipLaunchKernelGGL((int4_kernel<GATED, MB>), dim3((unsigned)(tiles < fit ? tiles : fit)), dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

template <bool GATED>
hipError_t launch_product(const Int4Args& g, hipStream_t stream) {
  return g.cap_rows <= 16 * (int64_t)g.E ? launch_tiles<GATED, 1>(g, stream) : launch_tiles<GATED, 2>(g, stream);
}

// ------------------------------------------------------------------------------------------------
// Rounding weights to 4 bits and reading them back: once, when weights are loaded.
// ------------------------------------------------------------------------------------------------

// A group's scale (rounded to bf16 first, the values are rounded against what is stored) and zero.
__device__ __forceinline__ uint16_t group_scale(float lo, float hi, bool bad, bool symmetric, float& divisor, float& zero) {
  const float range = symmetric ? fmaxf(-lo, hi) / 7.0f : (hi - lo) / 15.0f;
  const uint16_t s = bad ? (uint16_t)0x7FC0u : f32_to_bf16_bits(range);
  const float f = bf16_bits_to_f32(s);
  divisor = f > 0.0f && f < __builtin_inff() ? f : 1.0f;
  zero = symmetric ? 8.0f : (bad ? 0.0f : fminf(fmaxf(rintf(-lo / divisor), 0.0f), 15.0f));
  return s;
}

__device__ __forceinline__ uint32_t code(float w, float divisor, float zero, bool bad) {
  return bad ? 8u : (uint32_t)fminf(fmaxf(rintf(w / divisor) + zero, 0.0f), 15.0f);
}

// One thread a group of one row. `sk` and `sn`: pitches of the contraction and of the rows.
template <bool ROWS>
__global__ __launch_bounds__(kThreads) void int4_quantize_kernel(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                                 int E, int group, bool symmetric,
                                                                 uint8_t* __restrict__ q, uint16_t* __restrict__ scales,
                                                                 uint8_t* __restrict__ zeros) {
  const int64_t groups = (K + group - 1) / group, row_bytes = int4_row_bytes(K);
  const int64_t sk = ROWS ? 1 : N, sn = ROWS ? K : 1;
  const int64_t total = (int64_t)E * groups * N;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t n = i % N, gi = i / N % groups, e = i / (N * groups);
    const int64_t k0 = gi * group, k1 = k0 + group < K ? k0 + group : K;
    const uint16_t* p = w + e * N * K + n * sn;
    float lo = 0.0f, hi = 0.0f;
    bool bad = false;
    for (int64_t k = k0; k < k1; ++k) {
      const float v = bf16_bits_to_f32(p[k * sk]);
      lo = fminf(lo, v), hi = fmaxf(hi, v);
      bad = bad || !(fabsf(v) < __builtin_inff());
    }
    bad = bad || !(hi - lo < __builtin_inff());
    float divisor, zero;
    scales[i] = group_scale(lo, hi, bad, symmetric, divisor, zero);
    if (!symmetric) zeros[i] = (uint8_t)zero;
    uint8_t* out = q + (e * N + n) * row_bytes;
    // whole 16 bytes, zeros behind the last value
    for (int64_t k = k0; k < k1; k += 32) {
      u32x4 o = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (k + j < k1) o[j >> 3] |= code(bf16_bits_to_f32(p[(k + j) * sk]), divisor, zero, bad) << (4 * (j & 7));
      }
      *reinterpret_cast<u32x4*>(out + k / 2) = o;
    }
  }
}

// bf16 [E, N, K] of packed weights, 8 values a thread.
__global__ __launch_bounds__(kThreads) void int4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                   const uint16_t* __restrict__ scales,
                                                                   const uint8_t* __restrict__ zeros, int64_t N,
                                                                   int64_t K, int E, int group, uint16_t* __restrict__ w) {
  const int64_t groups = (K + group - 1) / group, row_bytes = int4_row_bytes(K), pieces = K / 8;
  const int64_t total = (int64_t)E * N * pieces;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
    const int64_t c = i % pieces, row = i / pieces, n = row % N, e = row / N;
    const int64_t at = (e * groups + c * 8 / group) * N + n;
    const uint32_t v = *reinterpret_cast<const uint32_t*>(q + row * row_bytes + c * 4);
    const float s = bf16_bits_to_f32(scales[at]);
    const int z = zeros != nullptr ? zeros[at] : 8;
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack_bf16x2(s * (float)((int)((v >> (8 * j)) & 15u) - z), s * (float)((int)((v >> (8 * j + 4)) & 15u) - z));
    *reinterpret_cast<u32x4*>(w + row * K + c * 8) = o;
  }
}

unsigned grid_of(int64_t items) {
  const int64_t blocks = (items + kThreads - 1) / kThreads, most = (int64_t)device_cu_count(current_device()) * 16;
  return (unsigned)(blocks < most ? blocks : most);
}

}  // namespace

hipError_t launch_int4_quantize(const uint16_t* w, bool w_out_in, int64_t d_in, int64_t d_out, int32_t E, int32_t group,
                                uint8_t* q, uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const int64_t items = (int64_t)E * ((d_in + group - 1) / group) * d_out;
  const bool symmetric = zeros == nullptr;
  if (w_out_in)
    hipLaunchKernelGGL((int4_quantize_kernel<true>), dim3(grid_of(items)), dim3(kThreads), 0, stream, w, d_out, d_in, E,
                       group, symmetric, q, scales, zeros);
  else
    hipLaunchKernelGGL((int4_quantize_kernel<false>), dim3(grid_of(items)), dim3(kThreads), 0, stream, w, d_out, d_in, E,
                       group, symmetric, q, scales, zeros);
  return hipGetLastError();
}

hipError_t launch_int4_dequantize(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, int64_t d_in,
                                  int64_t d_out, int32_t E, int32_t group, uint16_t* w, hipStream_t stream) {
  hipLaunchKernelGGL(int4_dequantize_kernel, dim3(grid_of((int64_t)E * d_out * (d_in / 8))), dim3(kThreads), 0, stream, q,
                     scales, zeros, d_out, d_in, E, group, w);
  return hipGetLastError();
}

hipError_t launch_int4_product(const uint16_t* x, const int32_t* perm, int32_t k, int64_t tokens, const int32_t* offsets,
                               const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, int32_t group, bool gated,
                               int64_t cap_rows, int64_t K, int64_t N, int32_t E, uint16_t* out, hipStream_t stream) {
  const Int4Args g = {x, perm, k, tokens, q, scales, zeros, group, gated ? 2 * N : N, N, K, offsets, E, cap_rows, out};
  return gated ? launch_product<true>(g, stream) : launch_product<false>(g, stream);
}

}  // namespace moe
