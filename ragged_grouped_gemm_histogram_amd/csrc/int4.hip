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
// a step (wide tiles exchange them through LDS). The weights are the second operand, so a lane ends with one weight
// row and four tokens of a product and needs one scale and one zero a group.

#include <cstddef>

#include "grouped.h"
#include "int4.h"

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

__device__ __forceinline__ float bf16_lo(uint32_t x) { return __builtin_bit_cast(float, x << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t x) { return __builtin_bit_cast(float, x & 0xFFFF0000u); }

// Eight weights of a dword as bf16 16 + q, in the order 0 4, 1 5, 2 6, 3 7: a shift and one and-or for two. (One operand
// of an instruction may be a constant or a scalar register, so the other constant is kept in a vector register.)
__device__ __forceinline__ bf16x8 unpack(uint32_t w, uint32_t sixteen) {
  constexpr uint32_t kBits = 0x00780078u;
  const u32x4 v = {((w << 3) & kBits) | sixteen, ((w >> 1) & kBits) | sixteen, ((w >> 5) & kBits) | sixteen,
                   ((w >> 9) & kBits) | sixteen};
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
constexpr int kUnit = kInt4Unit;
constexpr int kBlocks = kInt4Blocks;  // blocks of 16 weight rows of a tile

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
  // (an expert below E whatever the counts have wrapped to: a lane's first prefix is 0)
  const int in = __popcll(__ballot(lane < f.per && at < E && mine <= tile - base)) - 1;
  e = owner * f.per + in;
  begin = base + __builtin_amdgcn_readlane(mine, in);
}

// What a wave holds of one unit: 128 values of its 64 weight rows, and scales and zeros of the group that this lane's
// quarter has to load. A lane's four rows lie next to each other (gated: two gate rows and the two up rows that go with
// them), so one load brings their scales and one their zeros, and a lane ends with neighbouring columns.
struct Unit {
  u32x4 w[kBlocks];
  uint32_t s[2], z[2];
};

// Scales (two a word) and zeros (a byte each) of a lane's four rows.
struct Scales {
  uint32_t s[2], z;
};

// The groups' scales from the quarters that loaded them: of `half` 0 for a unit's steps 0 and 1, of 1 for 2 and 3; out[j]
// for the step's parity.
template <int GS>
__device__ __forceinline__ void spread_scales(const Scales& v, int half, Scales (&out)[2]) {
  auto one = [&](uint32_t x, uint32_t& a, uint32_t& b) {
    if constexpr (GS == 4) {
      a = b = x;
    } else {
      const auto h = __builtin_amdgcn_permlane32_swap(x, x, false, false);  // the wave's halves, each in both
      const uint32_t mine = half == 0 ? h[0] : h[1];
      if constexpr (GS == 2) {
        a = b = mine;
      } else {
        const auto q = __builtin_amdgcn_permlane16_swap(mine, mine, false, false);
        a = q[0], b = q[1];
      }
    }
  };
  one(v.s[0], out[0].s[0], out[1].s[0]);
  one(v.s[1], out[0].s[1], out[1].s[1]);
  one(v.z, out[0].z, out[1].z);
}

// A buffer resource of `bytes` from a uniform address on (2 GiB at most: offsets stay below).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(const void* base, int64_t bytes) {
  bytes = bytes < 0 ? 0 : (bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform_addr(base)), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}

// The 64 weight rows of a wave, through buffer resources that end with the expert's: what lies behind reads as zeros.
template <bool GATED, int GS>
struct WeightRows {
  static constexpr int kParts = GATED ? 2 : 1, kGroups = 4 / GS, kCols = GATED ? 32 : 64;
  __amdgpu_buffer_rsrc_t w[kParts];
  int64_t s0[kParts], s_left[kParts];  // first scale of the rows, scales from there to the expert's last
  uint32_t w_off, s_off, row_bytes;

  __device__ __forceinline__ void place(const Int4Args& g, int e, int64_t n0, int groups, int lane) {
    const int quarter = lane >> 4, first = (lane & 15) * (GATED ? 2 : 4);
    row_bytes = (uint32_t)int4_row_bytes(g.K);
    w_off = first * row_bytes + quarter * 16;
    s_off = (uint32_t)(quarter / GS) * (uint32_t)g.w_rows + first;
    n0 = int4_first_column(n0, g.N);
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int64_t r0 = n0 + p * g.N;
      w[p] = resource(g.q + ((int64_t)e * g.w_rows + r0) * row_bytes, int4_bytes_left(g.w_rows, r0, row_bytes));
      s0[p] = uniform_i64((int64_t)e * groups * g.w_rows + r0);
      s_left[p] = uniform_i64((int64_t)groups * g.w_rows - r0);
    }
  }

  __device__ __forceinline__ uint32_t block_at(int b, int u) const {
    return int4_block_at(GATED, b, u, row_bytes);
  }

  __device__ __forceinline__ void load(const Int4Args& g, Unit& d, int u) const {
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
      d.w[b] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(w[GATED ? b >> 1 : 0], w_off, block_at(b, u), 0));
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      const int64_t skip = (int64_t)u * kGroups * g.w_rows;
      const auto sr = resource(g.scales + s0[p] + skip, (s_left[p] - skip) * 2);
      const auto zr = resource(g.zeros + s0[p] + skip, g.zeros != nullptr ? s_left[p] - skip : 0);
      if constexpr (GATED) {
        d.s[p] = __builtin_amdgcn_raw_buffer_load_b32(sr, s_off * 2, 0, 0);
        d.z[p] = __builtin_amdgcn_raw_buffer_load_b16(zr, s_off, 0, 0);
      } else {
        const auto s = __builtin_amdgcn_raw_buffer_load_b64(sr, s_off * 2, 0, 0);
        d.s[0] = s[0], d.s[1] = s[1];
        d.z[0] = __builtin_amdgcn_raw_buffer_load_b32(zr, s_off, 0, 0), d.z[1] = 0;
      }
    }
  }
};

// What a step of a unit adds to a group's sums: acc of x (16 + q), xs of x.
template <int MB>
__device__ __forceinline__ void multiply_step(const bf16x8 (&xv)[MB], const uint32_t (&w)[kBlocks], uint32_t sixteen,
                                              const bf16x8& ones, f32x4_t (&acc)[kBlocks][MB], f32x4_t (&xs)[MB]) {
#pragma unroll
  for (int m = 0; m < MB; ++m) xs[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m], ones, xs[m], 0, 0, 0);
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const bf16x8 wv = unpack(w[b], sixteen);
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[b][m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m], wv, acc[b][m], 0, 0, 0);
  }
}

// At a group's end, sum += s (acc - (16 + z) xs).
template <int MB>
__device__ __forceinline__ void add_group(const Scales& now, const f32x4_t (&acc)[kBlocks][MB], const f32x4_t (&xs)[MB],
                                          f32x4_t (&sum)[kBlocks][MB]) {
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) {
    const float scale = b & 1 ? bf16_hi(now.s[b >> 1]) : bf16_lo(now.s[b >> 1]);
    const float c = 16.0f + (float)((now.z >> (8 * b)) & 0xFFu);
#pragma unroll
    for (int m = 0; m < MB; ++m) {
#pragma unroll
      for (int r = 0; r < 4; ++r) sum[b][m][r] = fmaf(scale, fmaf(-c, xs[m][r], acc[b][m][r]), sum[b][m][r]);
      asm volatile("" : "+v"(sum[b][m]));  // added here: put off to the next unit, it would hold all of acc
    }
  }
}

template <int MB>
__device__ __forceinline__ void clear_group(f32x4_t (&acc)[kBlocks][MB], f32x4_t (&xs)[MB]) {
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    xs[m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) acc[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
}

// sum += s (q - z) x over one unit in registers. tokens(s): the 8 values of this lane for step s, in the weights' order.
template <bool GATED, int GS, class Tokens>
__device__ __forceinline__ void multiply_unit(Unit& d, uint32_t no_zeros, const bf16x8& ones, Tokens tokens,
                                              f32x4_t (&sum)[kBlocks][1]) {
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) transpose_quarters(d.w[b]);
  const Scales mine = {{d.s[0], d.s[1]}, (GATED ? d.z[0] | d.z[1] << 16 : d.z[0]) | no_zeros};
  Scales sc[2];
  uint32_t sixteen = 0x41804180u;
  asm volatile("" : "+v"(sixteen));
  f32x4_t acc[kBlocks][1], xs[1];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if (s % 2 == 0 && (s == 0 || GS < 4)) spread_scales<GS>(mine, s / 2, sc);
    const bf16x8 xv[1] = {tokens(s)};
    const uint32_t w[kBlocks] = {d.w[0][s], d.w[1][s], d.w[2][s], d.w[3][s]};
    if (s % GS == 0) clear_group(acc, xs);
    multiply_step<1>(xv, w, sixteen, ones, acc, xs);
    if (s % GS == GS - 1) add_group<1>(sc[s & 1], acc, xs, sum);
    __builtin_amdgcn_sched_barrier(0);  // (a step's operands at a time: unpacked early, they would fill the registers)
  }
}

// A lane's columns of one token: four (gated: SiLU(v0) v2 and SiLU(v1) v3) from column `col` on.
template <bool GATED>
__device__ __forceinline__ void store_columns(const Int4Args& g, int64_t row, int64_t col, const f32x4_t& v) {
  if (col >= g.N) return;
  if constexpr (GATED) {
    float h[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) h[i] = v[i] * __builtin_amdgcn_rcpf(1.0f + __expf(-v[i])) * v[i + 2];
    *reinterpret_cast<uint32_t*>(g.out + row * g.N + col) = pack_bf16x2(h[0], h[1]);
  } else {
    *reinterpret_cast<u32x2_t*>(g.out + row * g.N + col) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// Few rows an expert: tiles of 16 rows by 64 weight rows, the contraction split into a range of units for each of the
// four waves, whose sums are joined through LDS. GS: steps of a group.
//
// What a call of few rows waits for is the chain offsets, tile, loads, join, so all of a unit's loads (weights,
// scales, zeros, tokens) go out together, the tile is found without a barrier, and as many waves are resident
// as the registers allow: four workgroups a CU. Measured: gate/up of 4 tokens, 32 of 128 experts of 2 x 768 x 2048
// in groups of 64 (53 MB) 16.4 us, the projection of the same tokens (27 MB) 10.3 us. Tried: the scales loaded when
// a group ends 24.1 and 13.8 us; a lane's rows 16 apart, so eight loads of scales and zeros and a join by columns,
// 18.2 and 10.6 us; the next unit's weights loaded before the products of this one 26.5 and 13.3 us (the registers
// for them spill, and loads return in order, so a spilled value waits for them too).
template <bool GATED, int GS>
__global__ __launch_bounds__(kThreads, 4) void int4_kernel(Int4Args g) {
  constexpr int BM = 16, kCols = GATED ? 32 : 64;
  __shared__ int offs[MOE_MAX_EXPERTS + 1], prefix[MOE_MAX_EXPERTS];
  __shared__ f32x4_t red[kWaves][4][64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int quarter = lane >> 4, r16 = lane & 15;
  const Finder find = find_setup<BM>(g.offsets, g.E, g.cap_rows, offs, prefix, lane);

  const int n_tiles = (int)((g.N + kCols - 1) / kCols);
  const int64_t total = (int64_t)find.total * n_tiles;
  const int K = (int)g.K;
  const uint32_t no_zeros = g.zeros != nullptr ? 0u : 0x08080808u;
  const int units = (K + kUnit - 1) / kUnit;
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

    // tokens past the last repeat the first, they are not stored
    int64_t row = row0 + (r16 < valid ? r16 : 0);
    if (g.perm != nullptr) row = clamp_row((int64_t)g.perm[row] / g.k, g.tokens - 1);
    const uint16_t* xr = g.x + row * g.K;
    WeightRows<GATED, GS> rows;
    rows.place(g, e, n0, groups, lane);
    f32x4_t sum[kBlocks][1];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) sum[b][0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int u = u_lo; u < u_hi; ++u) {
      Unit unit;
      rows.load(g, unit, u);
      u32x4 x[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int k = u * kUnit + s * 32 + quarter * 8;  // (behind the row's end: its last values, multiplied as zeros)
        x[s] = *reinterpret_cast<const u32x4*>(xr + (k < K ? k : K - 8));
      }
      multiply_unit<GATED, GS>(unit, no_zeros, ones, [&](int s) {
        return pair_up(u * kUnit + s * 32 + quarter * 8 < K ? x[s] : u32x4{0u, 0u, 0u, 0u});
      }, sum);
    }
    // Join the waves' parts: value r of a lane is token 4 (l / 16) + r; wave r adds those of all waves.
#pragma unroll
    for (int r = 0; r < 4; ++r) red[wave][r][lane] = f32x4_t{sum[0][0][r], sum[1][0][r], sum[2][0][r], sum[3][0][r]};
    __syncthreads();
    f32x4_t v = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) v += red[w][wave][lane];
    const int t = quarter * 4 + wave;
    if (t < valid) store_columns<GATED>(g, row0 + t, n0 + r16 * (kCols / 16), v);
    __syncthreads();
  }
}

// Workgroups a CU, as the grid counts them. LDS holds three with 32 rows in groups of 128 and, up to about 290 experts, of
// 64; in groups of 32, or with more experts, two, and the third starts when one of them is done.
constexpr int wide_resident(int mb) { return mb == 2 ? 3 : 2; }

// A unit of a wide tile in LDS, brought there by direct loads. Token row t's 16-byte piece c stands at c ^ (t % 16): 16
// rows' pieces of one c cover all banks. A weight row's quarters stand 256 bytes apart, so the 64 lanes of a step, which
// read one dword each, cover all banks too. Scales and zeros are the wave's 64 rows' (gated: 32 gate rows, 32 up rows).
template <int MB, int GS>
struct WideUnit {
  static constexpr int kGroups = 4 / GS;
  u32x4 tokens[16 * MB][16];
  uint32_t weights[kWaves][kBlocks][64][4];
  uint16_t scales[kWaves][kGroups][64];
  uint8_t zeros[kWaves][kGroups][64];
};

__device__ const u32x4 kZeros16 = {0u, 0u, 0u, 0u};  // what a token has behind its last value

// 16 bytes from each lane's address, 4 through a buffer resource, into LDS as dma16_buf.
__device__ __forceinline__ void dma16_at(const void* from, uint32_t lds_addr) {
  lds_addr = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off"
               :
               : "v"(from), "s"(lds_addr)
               : "memory", "m0");
}
__device__ __forceinline__ void dma4_buf(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint32_t lds_addr) {
  lds_addr = __builtin_amdgcn_readfirstlane(lds_addr);
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds"
               :
               : "v"(off), "s"(rsrc), "s"(lds_addr)
               : "memory", "m0");
}

// More rows an expert: tiles of 16 MB rows by 256 weight rows (gated: 128 columns' gate and up rows), 64 for each of the
// four waves over the whole contraction. One unit is multiplied while the next comes into LDS without passing registers.
// Bound by unpacking (about 250 vector operations a unit and wave, 40 matrix instructions, and as many again a
// group for its scales) and by how evenly the tiles fall on the CUs. Measured: gate/up of 256 tokens, top-8 of 64 experts,
// skewed, 2048 -> 2 x 768 45.6 us (narrow tiles 57); units through registers, loaded where they are needed, 49, and 39
// where this takes 35.7 with 32 rows for each expert. Tried: three or four units in LDS 36.7 us there, and 744 for
// 618 with 1024 rows (fewer workgroups a CU); a step unpacked between the matrix instructions of the one before 36.4 and
// 725 (its registers spill). With 64 rows 1 to 13 registers of the 256 spill as it is.
template <bool GATED, int MB, int GS>
__global__ __launch_bounds__(kThreads, wide_resident(MB)) void int4_wide_kernel(Int4Args g) {
  constexpr int BM = 16 * MB, kWaveCols = GATED ? 32 : 64, kCols = kWaves * kWaveCols;
  typedef WideUnit<MB, GS> Stage;
  extern __shared__ __attribute__((aligned(1024))) unsigned char lds[];
  const Stage* ring = reinterpret_cast<const Stage*>(lds);
  int *offs = reinterpret_cast<int*>(lds + 2 * sizeof(Stage)), *prefix = offs + g.E + 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int quarter = lane >> 4, r16 = lane & 15;
  const Finder find = find_setup<BM>(g.offsets, g.E, g.cap_rows, offs, prefix, lane);
  const int n_tiles = (int)((g.N + kCols - 1) / kCols);
  const int64_t total = (int64_t)find.total * n_tiles;
  const int K = (int)g.K;
  const uint32_t no_zeros = g.zeros != nullptr ? 0u : 0x08080808u;
  const int units = (K + kUnit - 1) / kUnit;
  const int groups = (K + 32 * GS - 1) / (32 * GS);
  const bf16x8 ones = __builtin_bit_cast(bf16x8, u32x4{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u});
  uint32_t sixteen = 0x41804180u;
  asm volatile("" : "+v"(sixteen));
  const uint32_t lds0 = (uint32_t)reinterpret_cast<uintptr_t>(lds);
  // what this lane brings of a unit: 8 values of one token row of 16, scales of 8 weight rows, zeros of 4
  const int slot = wave * 4 + quarter, value = ((lane & 15) ^ slot) * 8;
  const uint32_t s_row = GATED ? ((lane & 7) >> 2) * (uint32_t)g.N + (lane & 3) * 8 : (lane & 7) * 8;
  const uint32_t s_off = ((uint32_t)(lane >> 3) * (uint32_t)g.w_rows + s_row) * 2;
  const uint32_t z_row = GATED ? ((lane & 15) >> 3) * (uint32_t)g.N + (lane & 7) * 4 : (lane & 15) * 4;
  const uint32_t z_off = (uint32_t)(lane >> 4) * (uint32_t)g.w_rows + z_row;

  for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
    const uint32_t gm = (uint32_t)(tile / n_tiles);
    const int64_t n0 = (tile - (int64_t)gm * n_tiles) * kCols + wave * kWaveCols;
    int e;
    uint32_t begin;
    find_tile(find, g.E, gm, lane, e, begin);
    const int64_t lo = offs[e], hi = offs[e + 1];
    const int64_t row0 = lo + (int64_t)(gm - begin) * BM;
    if (row0 < lo || row0 >= hi) continue;  // wrapped counts
    const int valid = (int)(hi - row0 < BM ? hi - row0 : BM);

    const uint16_t* xr[MB];  // (tokens past the last repeat the first, they are not stored)
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int t = m * 16 + slot;
      int64_t row = row0 + (t < valid ? t : 0);
      if (g.perm != nullptr) row = clamp_row((int64_t)g.perm[row] / g.k, g.tokens - 1);
      xr[m] = g.x + row * g.K;
    }
    WeightRows<GATED, GS> rows;
    rows.place(g, e, n0, groups, lane);

    auto stage = [&](int u, int at) {
      const uint32_t to = lds0 + at * (uint32_t)sizeof(Stage);
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
        dma16_buf(rows.w[GATED ? b >> 1 : 0], rows.w_off, rows.block_at(b, u),
                  to + (uint32_t)offsetof(Stage, weights) + (wave * kBlocks + b) * 1024);
      const int64_t skip = (int64_t)u * Stage::kGroups * g.w_rows;
      const auto sr = resource(g.scales + rows.s0[0] + skip, (rows.s_left[0] - skip) * 2);
      const auto zr = resource(g.zeros + rows.s0[0] + skip, g.zeros != nullptr ? rows.s_left[0] - skip : 0);
      if (lane < 8 * Stage::kGroups)
        dma16_buf(sr, s_off, 0, to + (uint32_t)offsetof(Stage, scales) + wave * (Stage::kGroups * 128));
      if (lane < 16 * Stage::kGroups)
        dma4_buf(zr, z_off, to + (uint32_t)offsetof(Stage, zeros) + wave * (Stage::kGroups * 64));
      const int k = u * kUnit + value;
#pragma unroll
      for (int m = 0; m < MB; ++m)
        dma16_at(k < K ? static_cast<const void*>(xr[m] + k) : &kZeros16, to + (m * 16 + wave * 4) * 256);
    };

    f32x4_t sum[kBlocks][MB];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int m = 0; m < MB; ++m) sum[b][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    auto multiply = [&](const Stage& st) {
      u32x4 x[2][MB];
      uint32_t w[2][kBlocks];
      Scales sc[2];
      auto read = [&](int s) {
#pragma unroll
        for (int m = 0; m < MB; ++m) x[s & 1][m] = st.tokens[m * 16 + r16][(s * 4 + quarter) ^ r16];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) w[s & 1][b] = st.weights[wave][b][s * 16 + r16][quarter];
        if (s % GS == GS - 1) {
          Scales& v = sc[s & 1];
          const uint16_t* sp = st.scales[wave][s / GS];
          const uint8_t* zp = st.zeros[wave][s / GS];
          if constexpr (GATED) {
            v.s[0] = reinterpret_cast<const uint32_t*>(sp)[r16], v.s[1] = reinterpret_cast<const uint32_t*>(sp)[16 + r16];
            v.z = reinterpret_cast<const uint16_t*>(zp)[r16] | (uint32_t)reinterpret_cast<const uint16_t*>(zp)[16 + r16] << 16;
          } else {
            const u32x2_t two = reinterpret_cast<const u32x2_t*>(sp)[r16];
            v.s[0] = two[0], v.s[1] = two[1];
            v.z = reinterpret_cast<const uint32_t*>(zp)[r16];
          }
          v.z |= no_zeros;
        }
      };
      f32x4_t acc[kBlocks][MB], xs[MB];
      read(0);
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s < 3) read(s + 1);
        bf16x8 xv[MB];
#pragma unroll
        for (int m = 0; m < MB; ++m) xv[m] = pair_up(x[s & 1][m]);
        if (s % GS == 0) clear_group(acc, xs);
        multiply_step<MB>(xv, w[s & 1], sixteen, ones, acc, xs);
        if (s % GS == GS - 1) add_group<MB>(sc[s & 1], acc, xs, sum);
        __builtin_amdgcn_sched_barrier(0);  // (as in multiply_unit)
      }
    };

    stage(0, 0);
    for (int u = 0; u < units; ++u) {
      wait_vmcnt_lds<0>();
      bare_barrier();  // unit u is there, and the place of u - 1 is free
      if (u + 1 < units) stage(u + 1, (u + 1) & 1);
      multiply(ring[u & 1]);
    }
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = m * 16 + quarter * 4 + r;
        if (t < valid)
          store_columns<GATED>(g, row0 + t, n0 + r16 * (kWaveCols / 16),
                               f32x4_t{sum[0][m][r], sum[1][m][r], sum[2][m][r], sum[3][m][r]});
      }
    lds_barrier();  // (the ring's last reads, before the next tile's units)
  }
}

// Tiles of a call, as far as the host knows: each expert with rows ends with a tile that is half full on average.
double expected_tiles(const Int4Args& g, int rows, int cols) {
  const double experts = (double)(g.cap_rows < g.E ? g.cap_rows : g.E);
  const double by_rows = (double)g.cap_rows / rows + experts / 2;
  return (by_rows > experts ? by_rows : experts) * (double)((g.N + cols - 1) / cols);
}

// LDS of a wide tile with the tables of as many experts as there can be (the same for every call: two may run at once).
constexpr int kMostLds = 2 * (int)sizeof(WideUnit<4, 1>) + (2 * MOE_MAX_EXPERTS + 1) * (int)sizeof(int);

template <class Kernel>
hipError_t launch_tiles(Kernel kernel, const Int4Args& g, int rows, int cols, int resident, size_t lds, hipStream_t stream) {
  if (lds > 64 * 1024) {
    const hipError_t e =
        hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, kMostLds);
    if (e != hipSuccess) return e;
  }
  const int64_t most_experts = g.cap_rows < g.E ? g.cap_rows : g.E;
  const int64_t tiles = (g.cap_rows / rows + most_experts) * ((g.N + cols - 1) / cols);
  const int64_t fit = (int64_t)device_cu_count(current_device()) * resident;
  hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < fit ? tiles : fit)), dim3(kThreads), lds, stream, g);
  return hipGetLastError();
}

// The kind of tile whose estimated time in us is least. Narrow tiles (four resident a CU) wait 2.8 us for each unit of
// their longest wave; a wide one waits for each unit of the contraction, 1.2 us with 32 rows and 2.5 with 64, or as
// long as the tiles of a CU take to unpack, 1.0 and 1.65 us a tile. Over 90 calls (1 to 128 experts, 16 to 4096 rows, 64 to
// 3200 values by 64 to 3200 columns, even and skewed) the choice takes 0.5% longer than the best one in the mean, 14%
// at worst; by the mean of the rows per expert alone (up to 16, up to 48, above) it took 33% longer. 64 experts of
// 2048 -> 2 x 768 in groups of 128 with 16, 32, 64, 128 and 1024 rows each: 35, 36, 58, 90 and 618 us.
template <bool GATED, int GS>
hipError_t launch_rows(const Int4Args& g, hipStream_t stream) {
  constexpr int kOut = GATED ? 32 : 64;
  const double cus = (double)device_cu_count(current_device()), units = (double)((g.K + kUnit - 1) / kUnit);
  auto larger = [](double a, double b) { return a > b ? a : b; };
  const double longest = (double)(((g.K + kUnit - 1) / kUnit + kWaves - 1) / kWaves);
  const double narrow = larger(1.0, expected_tiles(g, 16, kOut) / (4 * cus)) * (1.0 + 2.8 * longest);
  const double wide32 = 3.0 + units * larger(1.2, 1.0 * expected_tiles(g, 32, 4 * kOut) / cus);
  const double wide64 = 2.7 + units * larger(2.5, 1.65 * expected_tiles(g, 64, 4 * kOut) / cus);
  if (narrow <= wide32 && narrow <= wide64) return launch_tiles(int4_kernel<GATED, GS>, g, 16, kOut, 4, 0, stream);
  const size_t tables = (2 * g.E + 1) * sizeof(int);
  if (wide32 <= wide64)
    return launch_tiles(int4_wide_kernel<GATED, 2, GS>, g, 32, 4 * kOut, wide_resident(2),
                        2 * sizeof(WideUnit<2, GS>) + tables, stream);
  return launch_tiles(int4_wide_kernel<GATED, 4, GS>, g, 64, 4 * kOut, wide_resident(4),
                      2 * sizeof(WideUnit<4, GS>) + tables, stream);
}

template <bool GATED>
hipError_t launch_product(const Int4Args& g, int group, hipStream_t stream) {
  return group == 32 ? launch_rows<GATED, 1>(g, stream)
                     : (group == 64 ? launch_rows<GATED, 2>(g, stream) : launch_rows<GATED, 4>(g, stream));
}

// ------------------------------------------------------------------------------------------------
// Rounding weights to 4 bits, once, when they are loaded, and reading them back, for calls of many rows. Bound by HBM
// and the exact quotients: 64 x 1536 x 2048 (503 MB read and written, 102 us at a copy's rate) 193 us, with the
// contraction outermost 205 us in groups of 32 and 314 in groups of 128; back 89 us.
// ------------------------------------------------------------------------------------------------

// A group's scale (rounded to bf16 first, the values are rounded against what is stored), the divisor (1 for a scale
// of 0) and the zero.
struct GroupCode {
  uint16_t scale;
  float divisor, zero;
  bool bad;
};

__device__ __forceinline__ GroupCode group_code(float lo, float hi, bool bad, bool symmetric) {
  GroupCode c;
  c.bad = bad || !(hi - lo < __builtin_inff());
  const float range = symmetric ? fmaxf(-lo, hi) / 7.0f : (hi - lo) / 15.0f;
  c.scale = c.bad ? (uint16_t)0x7FC0u : f32_to_bf16_bits(range);
  const float f = bf16_bits_to_f32(c.scale);
  c.divisor = f > 0.0f && f < __builtin_inff() ? f : 1.0f;
  c.zero = symmetric ? 8.0f : (c.bad ? 0.0f : fminf(fmaxf(rintf(-lo / c.divisor), 0.0f), 15.0f));
  return c;
}

__device__ __forceinline__ uint32_t code_of(float w, const GroupCode& c) {
  return c.bad ? 8u : (uint32_t)fminf(fmaxf(rintf(w / c.divisor) + c.zero, 0.0f), 15.0f);
}

template <int CTRL>
__device__ __forceinline__ int dpp(int x) {
  return __builtin_amdgcn_mov_dpp(x, CTRL, 0xF, 0xF, true);
}
template <int CTRL>
__device__ __forceinline__ void join_lanes(float& lo, float& hi, int& bad) {
  lo = fminf(lo, __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, lo))));
  hi = fmaxf(hi, __builtin_bit_cast(float, dpp<CTRL>(__builtin_bit_cast(int, hi))));
  bad |= dpp<CTRL>(bad);
}

// A workgroup's tile of stored weights: 32 rows by 512 values, a row to a wave at a time, 8 values a lane, so every
// access is whole lines; the scales and zeros, whose rows run the other way, go through LDS.
constexpr int kTileRows = 32, kTileK = 512, kTileGroups = kTileK / 32;
struct RowTile {
  int64_t e, n0, k0;
};
__device__ __forceinline__ RowTile row_tile(int64_t i, int64_t n_tiles, int64_t k_tiles) {
  const int64_t rest = i / k_tiles;
  return {rest / n_tiles, rest % n_tiles * kTileRows, i % k_tiles * kTileK};
}

__global__ __launch_bounds__(kThreads) void int4_quantize_rows_kernel(const uint16_t* __restrict__ w, int64_t N, int64_t K,
                                                                      int64_t E, int group, bool symmetric,
                                                                      uint8_t* __restrict__ q,
                                                                      uint16_t* __restrict__ scales,
                                                                      uint8_t* __restrict__ zeros) {
  __shared__ uint16_t s_tile[kTileGroups][kTileRows];
  __shared__ uint8_t z_tile[kTileGroups][kTileRows];
  const int64_t groups = (K + group - 1) / group, row_bytes = int4_row_bytes(K);
  const int64_t n_tiles = (N + kTileRows - 1) / kTileRows, k_tiles = (K + kTileK - 1) / kTileK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = group / 8;  // lanes of a group
  for (int64_t i = blockIdx.x; i < E * n_tiles * k_tiles; i += gridDim.x) {
    const RowTile t = row_tile(i, n_tiles, k_tiles);
    const int64_t k = t.k0 + lane * 8;
    for (int r = wave; r < kTileRows && t.n0 + r < N; r += kWaves) {
      const int64_t row = t.e * N + t.n0 + r;
      float v[8];
      u32x4 x = {0u, 0u, 0u, 0u};
      if (k < K) x = *reinterpret_cast<const u32x4*>(w + row * K + k);
      float lo = 0.0f, hi = 0.0f;
      int bad = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = j & 1 ? bf16_hi(x[j >> 1]) : bf16_lo(x[j >> 1]);
        lo = fminf(lo, v[j]), hi = fmaxf(hi, v[j]);
        bad |= !(fabsf(v[j]) < __builtin_inff());
      }
      join_lanes<0xB1>(lo, hi, bad);
      join_lanes<0x4E>(lo, hi, bad);
      if (per > 4) join_lanes<0x141>(lo, hi, bad);
      if (per > 8) join_lanes<0x140>(lo, hi, bad);
      const GroupCode c = group_code(lo, hi, bad != 0, symmetric);
      uint32_t o = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) o |= code_of(v[j], c) << (4 * j);
      // whole 16 bytes, zeros behind the last value
      if (k / 2 < row_bytes) *reinterpret_cast<uint32_t*>(q + row * row_bytes + k / 2) = k < K ? o : 0u;
      if (lane % per == 0) s_tile[lane / per][r] = c.scale, z_tile[lane / per][r] = (uint8_t)c.zero;
    }
    __syncthreads();
    for (int j = threadIdx.x; j < kTileK / group * kTileRows; j += kThreads) {
      const int gi = j / kTileRows, r = j % kTileRows;
      const int64_t g = t.k0 / group + gi;
      if (g < groups && t.n0 + r < N) {
        const int64_t at = (t.e * groups + g) * N + t.n0 + r;
        scales[at] = s_tile[gi][r];
        if (!symmetric) zeros[at] = z_tile[gi][r];
      }
    }
    __syncthreads();
  }
}

// Weights with the contraction outermost: a thread holds a group of two neighbouring columns, whose values it reads once.
template <int GROUP>
__global__ __launch_bounds__(kThreads) void int4_quantize_columns_kernel(const uint16_t* __restrict__ w, int64_t N,
                                                                         int64_t K, int64_t E, bool symmetric,
                                                                         uint8_t* __restrict__ q,
                                                                         uint16_t* __restrict__ scales,
                                                                         uint8_t* __restrict__ zeros) {
  const int64_t groups = (K + GROUP - 1) / GROUP, row_bytes = int4_row_bytes(K), pairs = N / 2;
  for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < E * groups * pairs; i += (int64_t)gridDim.x * kThreads) {
    const int64_t n = i % pairs * 2, g = i / pairs % groups, e = i / (pairs * groups);
    const uint16_t* p = w + (e * K + g * GROUP) * N + n;
    const int in = (int)(K - g * GROUP < GROUP ? K - g * GROUP : GROUP);  // values of the group
    uint32_t x[GROUP];
    float lo[2] = {0.0f, 0.0f}, hi[2] = {0.0f, 0.0f};
    bool bad[2] = {false, false};
#pragma unroll
    for (int k = 0; k < GROUP; ++k) x[k] = k < in ? *reinterpret_cast<const uint32_t*>(p + k * N) : 0u;
#pragma unroll
    for (int k = 0; k < GROUP; ++k) {
      const float v[2] = {bf16_lo(x[k]), bf16_hi(x[k])};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        lo[c] = fminf(lo[c], v[c]), hi[c] = fmaxf(hi[c], v[c]);
        bad[c] = bad[c] || !(fabsf(v[c]) < __builtin_inff());
      }
    }
    uint32_t s = 0, z = 0;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const GroupCode gc = group_code(lo[c], hi[c], bad[c], symmetric);
      s |= (uint32_t)gc.scale << (16 * c), z |= (uint32_t)gc.zero << (8 * c);
      uint8_t* out = q + (e * N + n + c) * row_bytes + g * (GROUP / 2);
#pragma unroll
      for (int k = 0; k < GROUP; k += 32) {
        if (k >= in) continue;
        u32x4 o = {0u, 0u, 0u, 0u};  // whole 16 bytes, zeros behind the last value
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float v = c == 0 ? bf16_lo(x[k + j]) : bf16_hi(x[k + j]);
          o[j >> 3] |= (k + j < in ? code_of(v, gc) : 0u) << (4 * (j & 7));
        }
        *reinterpret_cast<u32x4*>(out + k / 2) = o;
      }
    }
    const int64_t at = (e * groups + g) * N + n;
    *reinterpret_cast<uint32_t*>(scales + at) = s;
    if (!symmetric) *reinterpret_cast<uint16_t*>(zeros + at) = (uint16_t)z;
  }
}

// bf16 [E, N, K] of packed weights.
__global__ __launch_bounds__(kThreads) void int4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                   const uint16_t* __restrict__ scales,
                                                                   const uint8_t* __restrict__ zeros, int64_t N,
                                                                   int64_t K, int64_t E, int group,
                                                                   uint16_t* __restrict__ w) {
  __shared__ float s_tile[kTileGroups][kTileRows + 1], z_tile[kTileGroups][kTileRows + 1];
  const int64_t groups = (K + group - 1) / group, row_bytes = int4_row_bytes(K);
  const int64_t n_tiles = (N + kTileRows - 1) / kTileRows, k_tiles = (K + kTileK - 1) / kTileK;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t i = blockIdx.x; i < E * n_tiles * k_tiles; i += gridDim.x) {
    const RowTile t = row_tile(i, n_tiles, k_tiles);
    for (int j = threadIdx.x; j < kTileK / group * kTileRows; j += kThreads) {
      const int gi = j / kTileRows, r = j % kTileRows;
      const int64_t g = t.k0 / group + gi;
      if (g < groups && t.n0 + r < N) {
        const int64_t at = (t.e * groups + g) * N + t.n0 + r;
        s_tile[gi][r] = bf16_bits_to_f32(scales[at]);
        z_tile[gi][r] = zeros != nullptr ? (float)zeros[at] : 8.0f;
      }
    }
    __syncthreads();
    const int64_t k = t.k0 + lane * 8;
    if (k < K) {
#pragma unroll 4
      for (int r = wave; r < kTileRows; r += kWaves) {
        if (t.n0 + r >= N) break;
        const int64_t row = t.e * N + t.n0 + r;
        const uint32_t v = *reinterpret_cast<const uint32_t*>(q + row * row_bytes + k / 2);
        const float s = s_tile[lane * 8 / group][r], z = z_tile[lane * 8 / group][r];
        u32x4 o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = pack_bf16x2(s * ((float)((v >> (8 * j)) & 15u) - z), s * ((float)((v >> (8 * j + 4)) & 15u) - z));
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(w + row * K + k));
      }
    }
    __syncthreads();
  }
}

unsigned grid_of(int64_t workgroups, int per_cu) {
  const int64_t most = (int64_t)device_cu_count(current_device()) * per_cu;
  return (unsigned)(workgroups < most ? workgroups : most);
}

inline int64_t row_tiles(int64_t N, int64_t K, int64_t E) {
  return E * ((N + kTileRows - 1) / kTileRows) * ((K + kTileK - 1) / kTileK);
}

}  // namespace

hipError_t launch_int4_quantize(const uint16_t* w, bool w_out_in, int64_t d_in, int64_t d_out, int32_t E, int32_t group,
                                uint8_t* q, uint16_t* scales, uint8_t* zeros, hipStream_t stream) {
  const bool symmetric = zeros == nullptr;
  if (w_out_in) {
    hipLaunchKernelGGL(int4_quantize_rows_kernel, dim3(grid_of(row_tiles(d_out, d_in, E), 8)), dim3(kThreads), 0, stream, w,
                       d_out, d_in, E, group, symmetric, q, scales, zeros);
    return hipGetLastError();
  }
  const int64_t items = (int64_t)E * ((d_in + group - 1) / group) * (d_out / 2);
  const dim3 grid(grid_of((items + kThreads - 1) / kThreads, 8));
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(kThreads), 0, stream, w, d_out, d_in, E, symmetric, q, scales, zeros);
    return hipGetLastError();
  };
  return group == 32 ? run(int4_quantize_columns_kernel<32>)
                     : (group == 64 ? run(int4_quantize_columns_kernel<64>) : run(int4_quantize_columns_kernel<128>));
}

hipError_t launch_int4_dequantize(const uint8_t* q, const uint16_t* scales, const uint8_t* zeros, int64_t d_in,
                                  int64_t d_out, int32_t E, int32_t group, uint16_t* w, hipStream_t stream) {
  hipLaunchKernelGGL(int4_dequantize_kernel, dim3(grid_of(row_tiles(d_out, d_in, E), 8)), dim3(kThreads), 0, stream, q,
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
