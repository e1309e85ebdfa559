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
// a step. The weights are the second operand, so a lane ends with one weight row and four tokens: it needs
// one scale and one zero a group, which the quarters load one group each and then exchange.

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

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t cap) { return v < 0 ? 0 : (v > cap ? cap : v); }

// Which expert a row tile belongs to. Every wave finds it by itself, without a barrier: lane l adds up the
// tiles of `per` consecutive experts, a scan over the lanes gives where they begin, and the tables in LDS
// hold the same values whichever wave wrote them.
struct Finder {
  int* offs;    // [E + 1], clamped to the capacity
  int* prefix;  // [E], first row tile of each expert
  int per;
  uint32_t first, total;  // this lane's first tile, all tiles
};

template <int BM>
__device__ __forceinline__ Finder find_setup(const int32_t* offsets, int E, int64_t cap, int* offs, int* prefix, int lane) {
  Finder f;
  f.offs = offs, f.prefix = prefix, f.per = (E + 63) >> 6;
  const int e0 = lane * f.per;
  uint32_t sum = 0;  // (unsigned: offsets that are no running sum can wrap the counts)
  int lo = e0 < E ? (int)clamp_row(offsets[e0], cap) : 0;
  for (int i = 0; i < f.per; ++i) {
    const int e = e0 + i;
    if (e >= E) break;
    const int hi = (int)clamp_row(offsets[e + 1], cap);
    offs[e] = lo, prefix[e] = (int)sum;
    if (e == E - 1) offs[E] = hi;
    sum += hi > lo ? (uint32_t)(hi - lo + BM - 1) / BM : 0u;
    lo = hi;
  }
  uint32_t incl = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const uint32_t up = __shfl_up(incl, off, 64);
    if (lane >= off) incl += up;
  }
  f.first = incl - sum;
  f.total = __builtin_amdgcn_readlane(incl, 63);
  return f;
}

// Expert e and the first of its row tiles; tile < total.
__device__ __forceinline__ void find_tile(const Finder& f, int E, uint32_t tile, int lane, int& e, uint32_t& begin) {
  const int owner = __popcll(__ballot(f.first <= tile)) - 1;
  const uint32_t base = __builtin_amdgcn_readlane(f.first, owner);
  const int at = owner * f.per + (lane < f.per ? lane : f.per - 1);
  const uint32_t mine = at < E ? (uint32_t)f.prefix[at] : ~0u;
  const int in = __popcll(__ballot(lane < f.per && mine <= tile - base)) - 1;
  e = owner * f.per + in;
  begin = base + __builtin_amdgcn_readlane(mine, in);
}

// What a wave holds of one unit: 128 values of its weight rows and tokens, and the scale and zero of the group
// that this lane's quarter has to load.
template <int MB>
struct Unit {
  u32x4 w[kBlocks], x[MB][4];
  uint32_t s[kBlocks], z[kBlocks];
};

// A value that quarter j holds for group j of a unit (GS steps a group), as all lanes need it: out[j].
template <int GS>
__device__ __forceinline__ void spread_groups(uint32_t v, uint32_t (&out)[4 / GS]) {
  if constexpr (GS == 4) {
    out[0] = v;
  } else {
    const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // halves, each in both
    if constexpr (GS == 2) {
      out[0] = h[0], out[1] = h[1];
    } else {
      const auto a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
      const auto b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
      out[0] = a[0], out[1] = a[1], out[2] = b[0], out[3] = b[1];
    }
  }
}

// A buffer resource of `bytes` from a uniform address on (2 GiB at most: offsets stay below).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
  bytes = bytes < 0 ? 0 : (bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform_addr(base)), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// A tile: 16 MB rows by 64 weight rows (gated: 32 columns' gate and up rows), the contraction split into a
// range of units for each of the four waves, whose sums are joined through LDS. GS: steps of a group.
//
// What a call of few rows waits for is the chain offsets, tile, loads, join, so all of a unit's loads (weights,
// scales, zeros, tokens) go out together, the tile is found without a barrier, and as many waves are resident
// as the registers allow: four workgroups a CU (three with 32 rows). Measured: gate/up of 4 tokens, 32 of 128
// experts of 2 x 768 x 2048, groups of 64 19.1 us, the projection of the same tokens 11.1 us. Tried: scales read
// when a group ends 24.1 and 13.8 us; two units in flight a wave, which leaves three workgroups a CU, 18.8 and
// 19.4 us, the same at four workgroups with spilled registers 28.6 and 22.7 us.
template <bool GATED, int MB, int GS>
__global__ __launch_bounds__(kThreads, MB == 1 ? 4 : 3) void int4_kernel(Int4Args g) {
  constexpr int BM = 16 * MB, kCols = GATED ? 32 : 64, kGroups = 4 / GS;
  __shared__ int offs[MOE_MAX_EXPERTS + 1], prefix[MOE_MAX_EXPERTS];
  __shared__ __align__(16) float red[kWaves][kBlocks][MB][256];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int quarter = lane >> 4, r16 = lane & 15;
  const Finder find = find_setup<BM>(g.offsets, g.E, g.cap_rows, offs, prefix, lane);

  const int n_tiles = (int)((g.N + kCols - 1) / kCols);
  const int64_t total = (int64_t)find.total * n_tiles;
  const int K = (int)g.K;
  const uint32_t row_bytes = (uint32_t)int4_row_bytes(g.K);
  const int units = (K + kUnit - 1) / kUnit;
  const uint32_t no_zeros = g.zeros != nullptr ? 0u : 8u << 16;
  const int u_lo = units * wave / kWaves, u_hi = units * (wave + 1) / kWaves;
  const int groups = (K + 32 * GS - 1) / (32 * GS);
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});

  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const uint32_t gm = (uint32_t)(tile / n_tiles);
    const int n0 = (int)(tile - (int64_t)gm * n_tiles) * kCols;
    int e;
    uint32_t begin;
    find_tile(find, g.E, gm, lane, e, begin);
    const int64_t lo = offs[e], hi = offs[e + 1];
    const int64_t row0 = lo + (int64_t)(gm - begin) * BM;
    if (row0 < lo || row0 >= hi) continue;  // wrapped counts
    const int valid = (int)(hi - row0 < BM ? hi - row0 : BM);

    // Tokens past the last repeat the first, weight rows past the last read as zeros or as what stands there;
    // neither is stored.
    const uint16_t* xr[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int t = m * 16 + r16;
      int64_t row = row0 + (t < valid ? t : 0);
      if (g.perm != nullptr) row = clamp_row((int64_t)g.perm[row] / g.k, g.tokens - 1);
      xr[m] = g.x + row * g.K;
    }
    // Everything of the experts is read through buffer resources that end with the expert's rows: what lies
    // behind reads as zeros.
    constexpr int kParts = GATED ? 2 : 1;
    __amdgpu_buffer_rsrc_t wr[kParts];
    int64_t s0[kParts], s_left[kParts];  // first scale of the tile's rows, scales from there to the expert's last
    const uint32_t w_off = (uint32_t)r16 * row_bytes + quarter * 16;
    const uint32_t s_off = (uint32_t)(quarter / GS) * (uint32_t)g.w_rows + r16;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int64_t r0 = n0 + p * g.N;
      wr[p] = resource(g.q + ((int64_t)e * g.w_rows + r0) * row_bytes, (g.w_rows - r0) * row_bytes);
      s0[p] = uniform_i64((int64_t)e * groups * g.w_rows + r0);
      s_left[p] = uniform_i64((int64_t)groups * g.w_rows - r0);
    }

    auto load = [&](Unit<MB>& d, int u) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        const uint32_t at = w_off + (GATED ? b & 1 : b) * 16 * row_bytes + (uint32_t)u * 64;
        d.w[b] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr[GATED ? b >> 1 : 0], at, 0, 0));
      }
#pragma unroll
      for (int p = 0; p < kParts; ++p) {
        const int64_t skip = (int64_t)u * kGroups * g.w_rows;
        const auto sr = resource(g.scales + s0[p] + skip, (s_left[p] - skip) * 2);
        const auto zr = resource(g.zeros + s0[p] + skip, g.zeros != nullptr ? s_left[p] - skip : 0);
#pragma unroll
        for (int c = 0; c < kBlocks / kParts; ++c) {
          const int b = p * (kBlocks / kParts) + c;
          d.s[b] = __builtin_amdgcn_raw_buffer_load_b16(sr, (s_off + c * 16) * 2, 0, 0);
          d.z[b] = __builtin_amdgcn_raw_buffer_load_b8(zr, s_off + c * 16, 0, 0);
        }
      }
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int k = u * kUnit + s * 32 + quarter * 8;  // (behind the row's end: its last values, multiplied as zeros)
          d.x[m][s] = *reinterpret_cast<const u32x4*>(xr[m] + (k < K ? k : K - 8));
        }
    };

    f32x4_t sum[kBlocks][MB];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) sum[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](Unit<MB>& d, int u) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) transpose_quarters(d.w[b]);
      uint32_t sz[kBlocks][kGroups];  // scale in the low half, zero above
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) spread_groups<GS>(d.s[b] | d.z[b] << 16 | no_zeros, sz[b]);
      f32x4_t acc[kBlocks][MB], xs[MB];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        bf16x8 xv[MB];
        const bool in = u * kUnit + s * 32 + quarter * 8 < K;
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[m] = pair_up(in ? d.x[m][s] : u32x4{0u, 0u, 0u, 0u});
        if (s % GS == 0) {
#pragma unroll
          for (int m = 0; m < MB; ++m) {
            xs[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) acc[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
          }
        }
#pragma unroll
        for (int m = 0; m < MB; ++m) xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m], ones, xs[m], 0, 0, 0);
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const bf16x8 wv = unpack(d.w[b][s]);
#pragma unroll
          for (int m = 0; m < MB; ++m) acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m], wv, acc[b][m], 0, 0, 0);
        }
        if (s % GS == GS - 1) {
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const float scale = bf16_lo(sz[b][s / GS]), c = 16.0f + (float)(sz[b][s / GS] >> 16);
#pragma unroll
            for (int m = 0; m < MB; ++m)
#pragma unroll
              for (int r = 0; r < 4; ++r) sum[b][m][r] = fmaf(scale, fmaf(-c, xs[m][r], acc[b][m][r]), sum[b][m][r]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);  // (a step's operands at a time: unpacked early, they would fill the registers)
      }
    };

    for (int u = u_lo; u < u_hi; ++u) {
      Unit<MB> unit;
      load(unit, u);
      multiply(unit, u);
    }
    // Join the waves' parts: value r of lane l is token 4 (l / 16) + r and weight row l % 16, kept at 64 r + l, so
    // that lane l reads four consecutive columns of one token.
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) red[wave][b][m][64 * r + lane] = sum[b][m][r];
    __syncthreads();
    auto joined = [&](int b, int m) {
      f32x4_t v = *reinterpret_cast<const f32x4_t*>(&red[0][b][m][4 * lane]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) v += *reinterpret_cast<const f32x4_t*>(&red[w][b][m][4 * lane]);
      return v;
    };
    constexpr int kItems = (GATED ? 2 : 4) * MB;  // blocks of 16 tokens by 16 columns
    for (int i = wave; i < kItems; i += kWaves) {
      const int b = i / MB, m = i % MB;
      f32x4_t v = joined(b, m);
      if constexpr (GATED) {
        const f32x4_t up = joined(b + 2, m);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = v[r] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[r])) * up[r];
      }
      const int t = m * 16 + (lane >> 2 & 3) * 4 + (lane >> 4);
      const int64_t col = n0 + b * 16 + (lane & 3) * 4;
      if (t < valid && col < g.N)
        *reinterpret_cast<u32x2_t*>(g.out + (row0 + t) * g.N + col) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
    __syncthreads();
  }
}

template <bool GATED, int MB, int GS>
hipError_t launch_tiles(const Int4Args& g, hipStream_t stream) {
  constexpr int BM = 16 * MB;
  const int64_t n_tiles = (g.N + (GATED ? 31 : 63)) / (GATED ? 32 : 64);
  const int64_t most_experts = g.cap_rows < g.E ? g.cap_rows : g.E;
  const int64_t tiles = (g.cap_rows / BM + most_experts) * n_tiles;
  const int64_t fit = (int64_t)device_cu_count(current_device()) * (MB == 1 ? 4 : 3);
  hipLaunchKernelGGL((int4_kernel<GATED, MB, GS>), dim3((unsigned)(tiles < fit ? tiles : fit)), dim3(kThreads), 0, stream, g);
  return hipGetLastError();
}

template <bool GATED, int GS>
hipError_t launch_rows(const Int4Args& g, hipStream_t stream) {
  return g.cap_rows <= 16 * (int64_t)g.E ? launch_tiles<GATED, 1, GS>(g, stream) : launch_tiles<GATED, 2, GS>(g, stream);
}

template <bool GATED>
hipError_t launch_product(const Int4Args& g, int group, hipStream_t stream) {
  return group == 32 ? launch_rows<GATED, 1>(g, stream)
                     : (group == 64 ? launch_rows<GATED, 2>(g, stream) : launch_rows<GATED, 4>(g, stream));
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
  const Int4Args g = {x, perm, k, tokens, q, scales, zeros, gated ? 2 * N : N, N, K, offsets, E, cap_rows, out};
  return gated ? launch_product<true>(g, group, stream) : launch_product<false>(g, group, stream);
}

}  // namespace moe
