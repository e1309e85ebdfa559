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

#include <atomic>
#include <type_traits>

#include "grouped.h"
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
  uint16_t* out;            // [cap_rows, N], row pitch ldo
  int64_t ldo;
};

__device__ __forceinline__ i32x8 fp4_operand(const u32x4& v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

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

// ---------------------------------------------------------------------------------------------
// Many rows per expert: the pipelined tiles of the bf16 products. A stage is 256 values of every
// tile row, 128 bytes as there, four matrix steps of 64; the scale bytes of two stages (16 bytes a
// row) are loaded into LDS with the even one's values. A lane half takes the stage's chunks 4 half
// + step, so its four scale bytes are one LDS word and the step picks the byte.
// ---------------------------------------------------------------------------------------------
constexpr int kStageK = 256;

template <class C>
constexpr int kScaleBytes = 2 * (C::BM + C::BN) * 16;  // two pairs of stages

template <class C, bool KTAIL>
__global__ __launch_bounds__(C::THREADS) void mxfp4_pipe_kernel(MxGemmArgs g) {
  constexpr int BM = C::BM, BN = C::BN, NST = C::NST;
  constexpr int OPS = C::A_OPS + C::B_OPS;
  constexpr int S_LOADS = (BM + BN) / 64;  // wave loads of a stage pair's scales
  constexpr int S_OPS = (S_LOADS + C::NWAVES - 1) / C::NWAVES;
  static_assert(NST >= 2 && NST <= 3 && OPS * (NST - 1) < 64, "ring depth, vmcnt range");
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  __shared__ ProblemList<C::THREADS> pl;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  const int wm_u = __builtin_amdgcn_readfirstlane(wm);
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);

  build_problem_list<BM>(g, pl);
  const int total_mt = pl.mt_prefix[g.E];
  constexpr int TILE_N = C::GATED ? C::OUTW : BN;
  const int64_t n_tiles = (g.N + TILE_N - 1) / TILE_N;
  const int64_t total_tiles = (int64_t)total_mt * n_tiles;
  const int blocks = (int)mx_blocks(g.K);
  const int nk = (blocks + 7) / 8;
  const uint32_t qp = (uint32_t)mx_row_bytes(g.K), sp = (uint32_t)mx_scale_bytes(g.K);
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  unsigned char* const scale_lds = smem + C::LDS_BYTES;

  for (int64_t t = logical_worker(); t < total_tiles; t += gridDim.x) {
    const TileCoord tc = tile_coord<BM, TILE_N>(t, n_tiles, total_mt, g.E, pl);

    // Sources of each lane's 16-byte chunks, as byte offsets from wave-uniform bases (the host
    // guarantees that they fit). Rows past the expert's block and columns past N point at valid
    // ones: they only feed outputs that are never stored. The swizzle picks the chunk a lane fetches.
    const bool gather = g.a_rows != nullptr;
    auto a_row = [&](int r) -> uint32_t {  // row of a_q / a_s, from the base below
      const int rr = r < tc.rows_valid ? r : tc.rows_valid - 1;
      if (!gather) return (uint32_t)rr;
      const int32_t slot = g.a_rows[tc.row0 + rr];
      const uint32_t last = (uint32_t)(g.a_tokens * g.a_k) - 1u;
      return (slot < 0 ? 0u : min((uint32_t)slot, last)) / (uint32_t)g.a_k;
    };
    auto b_row = [&](int r) -> uint32_t {  // row of the expert's weights
      const int half = C::GATED && r >= BN / 2 ? 1 : 0;
      int64_t n = tc.n0 + (r - half * (BN / 2));
      if (n >= g.N) n = tc.n0;
      return (uint32_t)(n + half * g.N);
    };
    const int64_t a_first = gather ? 0 : tc.row0, b_first = (int64_t)tc.e * g.w_rows;
    const uint64_t a_base = uniform_addr(g.a_q + a_first * qp), b_base = uniform_addr(g.w_q + b_first * qp);
    const uint64_t as_base = uniform_addr(g.a_s + a_first * sp), bs_base = uniform_addr(g.w_s + b_first * sp);
    uint32_t a_off[C::A_OPS], b_off[C::B_OPS], s_off[S_OPS];
#pragma unroll
    for (int t2 = 0; t2 < C::A_OPS; ++t2) {
      const int r = 8 * (wave + C::NWAVES * t2) + (lane >> 3);
      a_off[t2] = a_row(r) * qp + swz(r, lane & 7) * 16;
    }
#pragma unroll
    for (int t2 = 0; t2 < C::B_OPS; ++t2) {
      const int r = 8 * (wave + C::NWAVES * t2) + (lane >> 3);
      b_off[t2] = b_row(r) * qp + swz(r, lane & 7) * 16;
    }
#pragma unroll
    for (int t2 = 0; t2 < S_OPS; ++t2) {
      const int r = 64 * (wave_u + C::NWAVES * t2) + lane;
      s_off[t2] = (r < BM ? a_row(r) : b_row(r - BM)) * sp;
    }
    // K not a multiple of 256: the last stage's chunks past the row get an offset past the buffer
    // resource's range and stage zeros. A lane fetches the same chunk of all its rows (they are
    // multiples of 8 apart with an even number of waves between).
    static_assert(C::NWAVES % 2 == 0, "rows of a lane are 16 apart or more");
    const bool in_tail = 8 * (nk - 1) + swz(8 * wave + (lane >> 3), lane & 7) < blocks;
    __amdgpu_buffer_rsrc_t a_rsrc, b_rsrc;
    if constexpr (KTAIL) {
      const int64_t a_range = gather ? g.a_tokens * qp : (int64_t)tc.rows_valid * qp;
      a_rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(a_base), (short)0, (int)a_range, 0x00020000);
      b_rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(b_base), (short)0, (int)(g.w_rows * qp), 0x00020000);
    }
    // Loads of stage kt, the ones with index % parts == part; an even stage's first part also
    // brings the scales of stages kt and kt + 1, before its values.
    auto issue_part = [&](int kt, int part, int parts) {
      const uint32_t sa = lds0 + (uint32_t)((kt % NST) * C::STAGE_BYTES);
      const uint32_t sb = sa + C::A_BYTES;
      const uint32_t wave_lds = __builtin_amdgcn_readfirstlane((uint32_t)wave * 1024u);
      if (part == 0 && (kt & 1) == 0) {
        const int pair = kt >> 1;
        const uint32_t sl = lds0 + C::LDS_BYTES + (uint32_t)((pair & 1) * (BM + BN) * 16);
#pragma unroll
        for (int t2 = 0; t2 < S_OPS; ++t2) {
          const int o = wave_u + C::NWAVES * t2;
          if (o < S_LOADS)
            dma16_off((o * 64 < BM ? as_base : bs_base) + (uint64_t)pair * 16, s_off[t2], sl + (uint32_t)o * 1024u);
        }
      }
      if constexpr (KTAIL) {
        const bool last = kt == nk - 1;
        const uint32_t soff = __builtin_amdgcn_readfirstlane((uint32_t)kt * 128u);
#pragma unroll
        for (int t2 = 0; t2 < C::A_OPS; ++t2)
          if (t2 % parts == part)
            dma16_buf(a_rsrc, last && !in_tail ? 0x80000000u : a_off[t2], soff, sa + wave_lds + (uint32_t)(C::NWAVES * t2 * 1024));
#pragma unroll
        for (int t2 = 0; t2 < C::B_OPS; ++t2)
          if (t2 % parts == part)
            dma16_buf(b_rsrc, last && !in_tail ? 0x80000000u : b_off[t2], soff, sb + wave_lds + (uint32_t)(C::NWAVES * t2 * 1024));
      } else {
        const uint64_t step = (uint64_t)kt * 128;
#pragma unroll
        for (int t2 = 0; t2 < C::A_OPS; ++t2)
          if (t2 % parts == part) dma16_off(a_base + step, a_off[t2], sa + wave_lds + (uint32_t)(C::NWAVES * t2 * 1024));
#pragma unroll
        for (int t2 = 0; t2 < C::B_OPS; ++t2)
          if (t2 % parts == part) dma16_off(b_base + step, b_off[t2], sb + wave_lds + (uint32_t)(C::NWAVES * t2 * 1024));
      }
    };
    auto issue = [&](int kt) { issue_part(kt, 0, 1); };

    f32x16 acc[C::FM][C::FN];
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    u32x4 af[2][C::FM], bfr[2][C::FN];  // fragments of a step: the one in use and the next
    int as[C::FM], bs[C::FN], as_next[C::FM], bs_next[C::FN];  // scale words of a stage, likewise
    auto load_frags = [&](int set, int slot, int ks) {
      const unsigned char* at = smem + slot * C::STAGE_BYTES;
      const unsigned char* bt = at + C::A_BYTES;
      const int chunk = 4 * (lane >> 5) + ks;
#pragma unroll
      for (int i = 0; i < C::FM; ++i) {
        const int r = wm * C::WTM + i * 32 + (lane & 31);
        af[set][i] = *reinterpret_cast<const u32x4*>(at + r * 128 + swz(r, chunk) * 16);
      }
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
        const int r = b_block_row<C>(wn, j) + (lane & 31);
        bfr[set][j] = *reinterpret_cast<const u32x4*>(bt + r * 128 + swz(r, chunk) * 16);
      }
    };
    auto load_scales = [&](int kt) {
      const unsigned char* st = scale_lds + ((kt >> 1) & 1) * (BM + BN) * 16 + (kt & 1) * 8 + (lane >> 5) * 4;
      // bytes past the row's last block may hold anything (255 is a NaN): their values are staged as
      // zeros, so a scale of 2^-127 keeps them zero
      uint32_t keep = 0xFFFFFFFFu;
      if constexpr (KTAIL) {
        const int left = blocks - 8 * kt - 4 * (lane >> 5);
        keep = left >= 4 ? keep : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
      }
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
        as_next[i] = (int)(*reinterpret_cast<const uint32_t*>(st + (wm * C::WTM + i * 32 + (lane & 31)) * 16) & keep);
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
        bs_next[j] = (int)(*reinterpret_cast<const uint32_t*>(st + (BM + b_block_row<C>(wn, j) + (lane & 31)) * 16) & keep);
    };
    auto take_scales = [&] {
#pragma unroll
      for (int i = 0; i < C::FM; ++i) as[i] = as_next[i];
#pragma unroll
      for (int j = 0; j < C::FN; ++j) bs[j] = bs_next[j];
    };
    auto mfmas = [&](int set, auto ks_c) {
      constexpr int ks = decltype(ks_c)::value;
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(bfr[set][j]), fp4_operand(af[set][i]),
                                                                      acc[i][j], 4, 4, ks, bs[j], ks, as[i]);
    };
    // Stage kt is complete for this wave once at most the later stages' values are in flight; after
    // the barrier it is complete for every wave, and every wave has read the stage before it.
    auto wait_stage = [&](int kt) {
      const int ahead = min(nk - 1, kt + NST - 2) - kt;
      if (NST >= 3 && ahead >= 1) wait_vmcnt_lds<(NST >= 3 ? 1 : 0) * OPS, true>();
      else wait_vmcnt_lds<0, true>();
      bare_barrier();
    };
    // tile start: every slot is free (the epilogue ended on a barrier)
    if constexpr (NST == 2) {
      issue(0);
      if (nk > 1) {
        issue(1);
        wait_vmcnt_lds<OPS, true>();
      } else {
        wait_vmcnt_lds<0, true>();
      }
      bare_barrier();
    } else {
#pragma unroll
      for (int s2 = 0; s2 < NST - 1; ++s2)
        if (s2 < nk) issue(s2);
      wait_stage(0);
    }
    if (wm_u * C::WTM >= tc.rows_valid) {
      // every row of this wave lies past the expert's block: its share of the loads and barriers only
      for (int kt = 0; kt + 1 < nk; ++kt) {
        if constexpr (NST >= 3) {
          if (kt + NST - 1 < nk) issue(kt + NST - 1);
        }
        wait_stage(kt + 1);
        if constexpr (NST == 2) {
          if (kt + 2 < nk) issue(kt + 2);
        }
      }
    } else {
      load_scales(0);
      load_frags(0, 0, 0);
      take_scales();
      auto stage = [&](int kt, auto last_c) {
        const int slot = kt % NST;
        if constexpr (NST >= 3) {
          if (kt + NST - 1 < nk) issue(kt + NST - 1);
        }
        load_frags(1, slot, 1);
        mfmas(0, std::integral_constant<int, 0>{});
        interleave_reads<C::FM * C::FN, C::FM + C::FN>();
        load_frags(0, slot, 2);
        mfmas(1, std::integral_constant<int, 1>{});
        interleave_reads<C::FM * C::FN, C::FM + C::FN>();
        load_frags(1, slot, 3);
        mfmas(0, std::integral_constant<int, 2>{});
        interleave_reads<C::FM * C::FN, C::FM + C::FN>();
        if constexpr (!decltype(last_c)::value) {
          wait_stage(kt + 1);
          if constexpr (NST == 2) {
            if (kt + 2 < nk) issue(kt + 2);
          }
          load_scales(kt + 1);
          load_frags(0, (kt + 1) % NST, 0);
        }
        mfmas(1, std::integral_constant<int, 3>{});
        if constexpr (!decltype(last_c)::value) take_scales();
      };
      for (int kt = 0; kt + 1 < nk; ++kt) stage(kt, std::false_type{});
      stage(nk - 1, std::true_type{});
    }
    lds_barrier();  // every wave is done with the ring before the epilogue reuses it
    epilogue<C, false>(acc, smem, g, tc);
  }
}

template <class C, bool KTAIL>
hipError_t launch_pipe(const MxGemmArgs& g, hipStream_t stream) {
  static std::atomic<bool> done[64] = {};
  auto kern = mxfp4_pipe_kernel<C, KTAIL>;
  constexpr int lds = C::LDS_BYTES + kScaleBytes<C>;
  const int dev = current_device();
  // Setting the attribute twice in a race of first calls is harmless.
  if (dev >= 0 && dev < 64 && !done[dev].load(std::memory_order_acquire)) {
    const hipError_t st = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (st != hipSuccess) return st;
    done[dev].store(true, std::memory_order_release);
  }
  constexpr int per_cu = 160 * 1024 / (lds + (int)sizeof(ProblemList<C::THREADS>));
  static_assert(per_cu >= 1, "the ring, the scales and the problem list must fit in LDS");
  hipLaunchKernelGGL(kern, dim3(device_cu_count(dev) * per_cu), dim3(C::THREADS), lds, stream, g);
  return hipGetLastError();
}

template <bool GATED>
using MxBig = std::conditional_t<GATED, Tile<256, 256, 4, 2, 2, true>, Tile<256, 256, 2, 4, 2, false>>;

template <bool GATED>
hipError_t launch_products(const MxGemmArgs& g, hipStream_t stream) {
  if (g.cap_rows == 0) return hipSuccess;
  const int cus = device_cu_count(current_device());
  // The pipelined tiles address values and scales by 32-bit offsets: from the tile's first row (gathered: the first
  // token), and from one expert's weights. Below 2 GiB also where offset 2^31 marks a chunk past the row.
  const int64_t qp = mx_row_bytes(g.K);
  const int64_t a_span = (g.a_rows != nullptr ? g.a_tokens : 256) * qp;
  const bool fits = a_span <= 0x7FFFFFFFll && g.w_rows * qp <= 0x7FFFFFFFll;
  if (fits && g.cap_rows >= (int64_t)64 * g.E) {
    if (g.K % kStageK != 0) return launch_pipe<MxBig<GATED>, true>(g, stream);
    return launch_pipe<MxBig<GATED>, false>(g, stream);
  }
  hipLaunchKernelGGL(mxfp4_thin_kernel<GATED>, dim3(cus * 4), dim3(kThinThreads), 0, stream, g);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_projection_mxfp4(const uint8_t* x_q, const uint8_t* x_s, const int32_t* offsets,
                                           const uint8_t* w_q, const uint8_t* w_s, int64_t cap_rows, int64_t d_in,
                                           int64_t d_out, int32_t E, uint16_t* y, hipStream_t stream) {
  const MxGemmArgs g{x_q, x_s, nullptr, 1, 0, w_q, w_s, d_out, d_out, d_in, offsets, E, cap_rows, y, d_out};
  return launch_products<false>(g, stream);
}

hipError_t launch_gemm_up_swiglu_mxfp4(const uint8_t* x_q, const uint8_t* x_s, int64_t x_rows, const int32_t* perm,
                                       int32_t k, const int32_t* offsets, const uint8_t* w_q, const uint8_t* w_s,
                                       int64_t cap_rows, int64_t d, int64_t h, int32_t E, uint16_t* h_buf,
                                       hipStream_t stream) {
  const MxGemmArgs g{x_q, x_s, perm, k, x_rows, w_q, w_s, 2 * h, h, d, offsets, E, cap_rows, h_buf, h};
  return launch_products<true>(g, stream);
}

}  // namespace moe
