// Grouped products of MXFP4 rows with MXFP4 expert weights, fp32 accumulation:
//
//   plain:  y[rows_e] = bf16( X_e W_e^T )                        W_e [N, K]
//   gated:  h[rows_e] = bf16( SiLU(g) * u ), [g | u] = X_e W_e^T   W_e [2N, K], gate rows first
//
// Every product of two 4-bit values and their blocks' powers of two that is a normal fp32 number is
// exact; sums are fp32, and there is one rounding, of the result (the gated form takes SiLU of the fp32 sums).
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
  uint8_t* out_q = nullptr;  // gated, instead of out: the result's MXFP4 rows
  uint8_t* out_s = nullptr;
};

__device__ __forceinline__ i32x8 fp4_operand(const u32x4& v) {
  return i32x8{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t cap) { return v < 0 ? 0 : (v > cap ? cap : v); }

// ---------------------------------------------------------------------------------------------
// Few rows per expert, or few tiles: 32 rows by 64 weight rows a workgroup, operands straight from memory to
// registers, the contraction split over the four waves and joined through LDS. Such a call is bound
// by reading the weights of the experts that have rows: a wave asks for BATCH units of 128 values
// before it multiplies them, the weights first, since they do not wait for the dispatch order, and
// four workgroups share a CU.
//
// Measured: gate/up of 4 tokens, 32 of 128 experts of 2 x 768 x 2048 (53 MB), 18.9 us with the weights of 24
// layers in turn, so from HBM, 15.7 us with one layer's again and again, so from the last-level cache. About
// 5.5 us pass whatever the size (offsets, prefix, first load, join); from HBM the rest runs at 4.0 TB/s (16
// tokens, all 128 experts, 214 MB: 58.5 us). The projection of the same tokens (27 MB) 12.6 and 10.0 us. Tried, from
// HBM and from cache: batches of 1 19.6 and 16.4 us (the projection 12.3 and 9.5), of 4 with two workgroups
// a CU 25.3 and 21.7, non-temporal weight loads 24.1 and 22.8 (a line is read by several loads). From
// cache alone, 16.2 us at the time: 16 x 16 x 128 products (64 consecutive bytes a row and load) 16.7 us and
// 44 instead of 31 us at 2048 rows; 8 waves 17.2 us.
// ---------------------------------------------------------------------------------------------
constexpr int kThinThreads = 256;
constexpr int kThinWaves = 4;
constexpr int kUnit = 128;  // contraction per step: four blocks, two per lane half
template <bool GATED>
constexpr int kThinCols = GATED ? 32 : 64;  // output columns of a tile

template <bool GATED, bool QUANT, int BATCH>
__global__ __launch_bounds__(kThinThreads, 4) void mxfp4_thin_kernel(MxGemmArgs g) {
  __shared__ int mt_prefix[MOE_MAX_EXPERTS + 1];
  __shared__ int offs[MOE_MAX_EXPERTS + 1];  // clamped to the capacity
  __shared__ uint32_t wave_total[kThinWaves];
  __shared__ float4 red[kThinWaves * 4 * 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 31, hh = lane >> 5;

  // prefix of the experts' 32-row tile counts
  {
    constexpr int kPer = MOE_MAX_EXPERTS / kThinThreads;
    uint32_t mt[kPer], sum = 0;  // (unsigned: offsets that are no running sum can wrap the counts)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid + i * kThinThreads;
      if (e <= g.E) offs[e] = (int)clamp_row(g.offsets[e], g.cap_rows);
    }
    if (tid == 0 && g.E == MOE_MAX_EXPERTS) offs[g.E] = (int)clamp_row(g.offsets[g.E], g.cap_rows);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      mt[i] = e < g.E ? mx_row_tiles(offs[e], offs[e + 1], 32) : 0u;
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
      if (e <= g.E) mt_prefix[e] = (int)run;
      run += mt[i];
    }
    if (tid == kThinThreads - 1 && g.E == MOE_MAX_EXPERTS) mt_prefix[g.E] = (int)run;
    __syncthreads();
  }
  constexpr int kCols = kThinCols<GATED>;
  const int n_tiles = (int)((g.N + kCols - 1) / kCols);
  const int64_t total = (int64_t)mt_prefix[g.E] * n_tiles;
  const int64_t qp = mx_row_bytes(g.K), sp = mx_scale_bytes(g.K);
  const int blocks = (int)mx_blocks(g.K);
  const int units = (int)((g.K + kUnit - 1) / kUnit);
  const int u_lo = units * wave / kThinWaves, u_hi = units * (wave + 1) / kThinWaves;
  const int b_end = min(blocks, 4 * u_hi);

  for (int64_t t = blockIdx.x; t < total; t += gridDim.x) {
    const int gm = (int)(t / n_tiles);
    const int n0 = (int)(t - (int64_t)gm * n_tiles) * kCols;
    int e = 0, hi_e = g.E;  // largest e with mt_prefix[e] <= gm
    while (hi_e - e > 1) {
      const int mid = (e + hi_e) >> 1;
      if (mt_prefix[mid] <= gm) e = mid; else hi_e = mid;
    }
    const int64_t lo = offs[e], hi = offs[e + 1];
    const int64_t row0 = lo + ((int64_t)gm - mt_prefix[e]) * 32;
    if (row0 < lo || row0 >= hi) continue;  // wrapped counts
    const int valid = (int)(hi - row0 < 32 ? hi - row0 : 32);
    // sources: rows past the block repeat its last, columns past N the tile's first; neither is stored
    int64_t a_row = row0 + (r < valid ? r : valid - 1);
    int32_t slot = 0;
    if (g.a_rows != nullptr) slot = g.a_rows[a_row];
    // weights through buffer resources that end with the tile's 32 rows: a block past this wave's part
    // gets an offset past the range and reads as zeros, with no branch between the loads
    __amdgpu_buffer_rsrc_t w_q[2], w_s[2];
    uint32_t w_row[2];
    const int64_t w_first = (int64_t)e * g.w_rows + n0;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int64_t left = g.N - n0 - (GATED ? 0 : f * 32);  // columns of this half; none: the other's again
      const int64_t row = w_first + (GATED ? f * g.N : (left > 0 ? f * 32 : 0));
      w_q[f] = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform_addr(g.w_q + row * qp)), (short)0,
                                                 (int)(32 * qp), 0x00020000);
      w_s[f] = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(uniform_addr(g.w_s + row * sp)), (short)0,
                                                 (int)(32 * sp), 0x00020000);
      w_row[f] = r < left ? (uint32_t)r : 0u;
    }
    f32x16 acc[2];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][i] = acc[1][i] = 0.f;
    for (int u0 = u_lo; u0 < u_hi; u0 += BATCH) {
      u32x4 av[BATCH][2], wv[BATCH][2][2];
      uint32_t as[BATCH], ws[BATCH][2];
      // blocks b and b + 1 of unit u0 + x, values and scale bytes
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const int b = 4 * (u0 + x) + 2 * hh;
#pragma unroll
        for (int f = 0; f < 2; ++f) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            wv[x][f][i] = __builtin_amdgcn_raw_buffer_load_b128(
                w_q[f], b + i < b_end ? w_row[f] * (uint32_t)qp + (uint32_t)(b + i) * 16u : 0x80000000u, 0, 0);
          ws[x][f] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(
              w_s[f], b < b_end ? w_row[f] * (uint32_t)sp + (uint32_t)b : 0x80000000u, 0, 0);
        }
      }
      if (u0 == u_lo && g.a_rows != nullptr) {
        const int64_t last = g.a_tokens * g.a_k - 1;
        a_row = (slot < 0 ? 0u : (uint32_t)(slot > last ? last : slot)) / (uint32_t)g.a_k;
      }
      // the row's blocks past the part are its last one again, times the weights' zeros
      const uint8_t* a_q = g.a_q + a_row * qp;
      const uint8_t* a_s = g.a_s + a_row * sp;
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        const int b = 4 * (u0 + x) + 2 * hh;
#pragma unroll
        for (int i = 0; i < 2; ++i) av[x][i] = *reinterpret_cast<const u32x4*>(a_q + min(b + i, b_end - 1) * 16);
        as[x] = *reinterpret_cast<const uint16_t*>(a_s + min(b, (b_end - 1) & ~1));
      }
#pragma unroll
      for (int x = 0; x < BATCH; ++x) {
        // bytes past the row's last block may hold anything (255 is a NaN)
        const int b = 4 * (u0 + x) + 2 * hh;
        const uint32_t keep = b + 1 < blocks ? 0xFFFFu : (b < blocks ? 0xFFu : 0u);
        const int a = (int)(as[x] & keep);
#pragma unroll
        for (int f = 0; f < 2; ++f) {
          const int w = (int)(ws[x][f] & keep);
          acc[f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(wv[x][f][0]), fp4_operand(av[x][0]), acc[f], 4,
                                                                   4, 0, w, 0, a);
          acc[f] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(wv[x][f][1]), fp4_operand(av[x][1]), acc[f], 4,
                                                                   4, 1, w, 1, a);
        }
      }
    }
    // the waves' sums, in wave order, one half after the other
    float4 sum[2];
#pragma unroll
    for (int f = 0; f < 2; ++f) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(wave * 4 + q) * 64 + lane] = float4{acc[f][4 * q], acc[f][4 * q + 1], acc[f][4 * q + 2], acc[f][4 * q + 3]};
      __syncthreads();
      sum[f] = red[wave * 64 + lane];  // this thread's quad of columns: q = wave
#pragma unroll
      for (int w = 1; w < kThinWaves; ++w) {
        const float4 v = red[(w * 4 + wave) * 64 + lane];
        sum[f].x += v.x; sum[f].y += v.y; sum[f].z += v.z; sum[f].w += v.w;
      }
      __syncthreads();  // red is reused
    }
    const int col = n0 + 8 * wave + 4 * hh;
    if constexpr (QUANT) {
      // the tile's 32 columns are one block a row: its bf16 rows go through LDS to four lanes a row
      uint2* h = reinterpret_cast<uint2*>(red);  // [32 rows][8 pieces of 4 columns]
      h[r * 8 + 2 * wave + hh] = col < g.N ? uint2{pack_bf16x2(swiglu(sum[0].x, sum[1].x), swiglu(sum[0].y, sum[1].y)),
                                                   pack_bf16x2(swiglu(sum[0].z, sum[1].z), swiglu(sum[0].w, sum[1].w))}
                                           : uint2{0u, 0u};
      __syncthreads();
      const int row = tid >> 2, piece = tid & 3;
      if (tid < 128 && row < valid) {
        const u32x4 v = reinterpret_cast<const u32x4*>(red)[row * 4 + piece];
        uint32_t top = max_magnitude(v);
        top = max(top, quad_xor<0xB1>(top));
        top = max(top, quad_xor<0x4E>(top));
        const uint32_t byte = scale_byte(top);
        const int64_t out_row = row0 + row, osp = mx_scale_bytes(g.N);
        reinterpret_cast<uint32_t*>(g.out_q + out_row * mx_row_bytes(g.N) + n0 / 2)[piece] = to_fp4(v, byte);
        uint8_t* os = g.out_s + out_row * osp;
        if (piece == 0) os[n0 / 32] = (uint8_t)byte;
        if (n0 + 32 >= g.N)  // the padding behind the last block
          for (int64_t z = n0 / 32 + 1 + piece; z < osp; z += 4) os[z] = 0;
      }
      __syncthreads();
    } else if (r < valid) {
      uint16_t* dst = g.out + (row0 + r) * g.N;
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
  }
}

// ---------------------------------------------------------------------------------------------
// Many rows per expert: 256 x 256 tiles on 8 waves, persistent workgroups, direct global -> LDS
// loads into a ring of four stages. A stage is 128 values of every tile row (64 bytes), two matrix
// steps of 64; the scale bytes of four stages (16 bytes a row) come with the first one's values. A
// lane half takes the stage's chunks 2 half + step, so its two scale bytes are neighbours and the
// step picks the byte.
//
// The ring runs on across tiles: while a tile's last stages are multiplied, the next tile's first
// four are loaded, and the results leave from registers (exchanges between lanes make whole lines)
// instead of through the ring's memory, so the loads of a new tile have no gap before them.
//
// Measured: gate/up of 8192 tokens, top-8 of 64 experts 2048 -> 2 x 768, skewed (392 GFLOP) 129 to 139 us from
// one card to the next; down projection of 65536 rows 768 -> 2048 of the same experts (206 GFLOP, 268 MB written) 87
// to 94 us; 16 experts 4096 -> 4096, 65536 rows, 3.5 PFLOP/s. The matrix unit is busy 37 and 28% of 279 and 198
// thousand cycles (the first two). What the rest is, in thousand cycles: 241 and 135 without SwiGLU and stores, 243
// and 160 without loads, 232 and 188 without LDS reads, 160 and 99 with products and barriers alone, 11 of them
// before the first product. So the down projection is bound by its stores, which HBM alone takes 120
// thousand cycles to write and which overlap half with the next tile's products, gate/up by LDS, loads and
// matrix unit sharing a stage. Tried and slower: 128 x 128 tiles, two workgroups a CU (gate/up 220, down
// 153 us when these were 150 and 114; over 170 random calls 0.3% would be gained by taking them where they
// win); four waves of 128 x 128 (registers spill); staggered starts; ordinary stores (106 us); wave
// priorities; products skipped by waves without rows.
// ---------------------------------------------------------------------------------------------
constexpr int kStageK = 128;
constexpr int kRing = 4;          // stages in LDS
constexpr int kGroup = 4;         // stages a row's 16 scale bytes cover
constexpr int kScaleRing = 3;     // scale groups in LDS: the last two of a tile and the next tile's first
// Row tiles of a group: the 32 tiles that an XCD's CUs run together are then 4 x 8. Gate/up of 8192 tokens, top-4 of 16
// experts 2880 -> 2 x 2880: 360 us with 4 (2: 360, 8: 374, 16: 378, 32: 386); the 64-expert products within 1%.
constexpr int kGroupRows = 4;
constexpr int kTableTiles = 64;   // tiles of a workgroup whose coordinates are worked out together

template <int BM_, int BN_, int WGM_, int WGN_, bool GATED_>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_;
  static constexpr bool GATED = GATED_;
  static constexpr int NWAVES = WGM * WGN, THREADS = 64 * NWAVES;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int OUTW = GATED ? BN / 2 : BN;
  static constexpr int A_BYTES = BM * 64, B_BYTES = BN * 64, STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int SCALE_BYTES = (BM + BN) * 16;
  static constexpr int LDS_BYTES = kRing * STAGE_BYTES + kScaleRing * SCALE_BYTES;
  static constexpr int A_OPS = BM / 16 / NWAVES, B_OPS = BN / 16 / NWAVES;  // wave loads of 16 rows
  static constexpr int S_OPS = (BM + BN) / 64 / NWAVES;                     // wave loads of 64 rows' scales
  static_assert(BM % (16 * NWAVES) == 0 && BN % (16 * NWAVES) == 0 && (BM + BN) % (64 * NWAVES) == 0 && BM % 64 == 0,
                "loads split evenly over the waves");
};

struct MxProblems {
  int mt_prefix[MOE_MAX_EXPERTS + 1];
  uint32_t wave_total[8];
  int4 table[kTableTiles];  // expert, first row, rows, first column
};

struct MxCoord {
  int e, row0, rows_valid, n0;
};

// Exchanges a lane bit (0 or 1: CTRL is the quad permute that flips it, `set` where it is set) with the
// choice between two registers, for four pairs: lanes that have it set take b of their partner into a, the
// others a of theirs into b.
template <int CTRL>
__device__ __forceinline__ void swap_bit(uint32_t (&a)[4], uint32_t (&b)[4], bool set) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const uint32_t from_b = quad_xor<CTRL>(b[w]), from_a = quad_xor<CTRL>(a[w]);  // read in every lane, whichever it keeps
    a[w] = set ? from_b : a[w];
    b[w] = set ? b[w] : from_a;
  }
}

// Accumulators to bf16 rows. acc[i][j][4 q + s] is row wm * WTM + 32 i + lane % 32, column (block
// column base + 8 q + 4 (lane / 32) + s). Three exchanges between lanes gather a row's 64 columns from
// the registers of one lane pair into eight lanes: the halves exchange the column block, lane bits 0 and
// 1 the group of 8 columns (q). Every store then writes 8 rows of 128 consecutive bytes, neighbouring
// lanes neighbouring bytes: a CU takes such stores at 110 bytes a cycle, those of the same lines with
// rows in the low lane bits at 32 (65536 x 2048 results of 768 values: 88 and 96 us a call). Rows past the block and columns past N fall outside the buffer
// resource and are dropped; every wave issues all its stores.
//
// QUANT: the rows leave as MXFP4. After the first exchange a lane holds a whole block of its row, so the
// block's maximum needs no other lane, and the lane stores its 16 bytes; the lower half's lanes store their
// row's two scale bytes.
template <class C, bool QUANT>
constexpr int kTileStores = C::FM * (QUANT ? 2 : 4) * (C::OUTW / C::WGN / 64);

template <class C, bool QUANT>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[C::FM][C::FN], const MxGemmArgs& g, const MxCoord& tc) {
  constexpr int kPieces = C::OUTW / C::WGN / 64;  // of 64 columns
  static_assert(C::OUTW / C::WGN % 64 == 0, "a wave stores whole lines");
  const int tid = epilogue_tid<true>(), lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  static_assert(!QUANT || (C::GATED && kPieces == 1), "quantised output is the gated projection's");
  __amdgpu_buffer_rsrc_t rsrc, s_rsrc;
  uint32_t row_bytes, s_bytes = 0;
  if constexpr (QUANT) {
    row_bytes = (uint32_t)mx_row_bytes(g.N);
    s_bytes = (uint32_t)mx_scale_bytes(g.N);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(g.out_q + (int64_t)tc.row0 * row_bytes, (short)0,
                                             (int)((uint32_t)tc.rows_valid * row_bytes), 0x00020000);
    s_rsrc = __builtin_amdgcn_make_buffer_rsrc(g.out_s + (int64_t)tc.row0 * s_bytes, (short)0,
                                               (int)((uint32_t)tc.rows_valid * s_bytes), 0x00020000);
  } else {
    row_bytes = (uint32_t)(g.ldo * 2);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(g.out + (int64_t)tc.row0 * g.ldo, (short)0,
                                             (int)((int64_t)tc.rows_valid * g.ldo * 2), 0x00020000);
  }
  const uint32_t row = (uint32_t)(wm * C::WTM + (lane & (QUANT ? 31 : 28)));
#pragma unroll
  for (int p = 0; p < kPieces; ++p) {
    const int64_t col = tc.n0 + (wn * kPieces + p) * 64 + 32 * (lane >> 5) + (QUANT ? 0 : 8 * (lane & 3));
    const uint32_t base = col < g.N ? row * row_bytes + (uint32_t)(QUANT ? col / 2 : col * 2) : 0x80000000u;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      uint32_t v[4][4];  // [group of 8 columns; after the exchanges: row lane & 28 + this][16 bytes]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t pk[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float f[4];
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            if constexpr (C::GATED) f[s] = swiglu(acc[i][2 * p + j][4 * q + s], acc[i][2 * kPieces + 2 * p + j][4 * q + s]);
            else f[s] = acc[i][2 * p + j][4 * q + s];
          }
          pk[j][0] = pack_bf16x2(f[0], f[1]);
          pk[j][1] = pack_bf16x2(f[2], f[3]);
        }
        // halves: the lower one gets the first column block's 8 columns, the upper one the second's
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const auto x = __builtin_amdgcn_permlane32_swap(pk[0][w], pk[1][w], false, false);
          v[q][w] = x[0];
          v[q][2 + w] = x[1];
        }
      }
      if constexpr (QUANT) {
        u32x4 part[4], out;
        uint32_t top = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          part[q] = u32x4{v[q][0], v[q][1], v[q][2], v[q][3]};
          if (col + 8 * q >= g.N) part[q] = u32x4{0u, 0u, 0u, 0u};  // a block that N cuts is filled with zeros
          top = max(top, max_magnitude(part[q]));
        }
        const uint32_t byte = scale_byte(top);
#pragma unroll
        for (int q = 0; q < 4; ++q) out[q] = to_fp4(part[q], byte);
        __builtin_amdgcn_raw_buffer_store_b128(out, rsrc, base + (uint32_t)(32 * i) * row_bytes, 0, 0);
        const auto both = __builtin_amdgcn_permlane32_swap(byte, byte, false, false);
        const uint32_t s_at = (row + (uint32_t)(32 * i)) * s_bytes + (uint32_t)((tc.n0 + wn * 64) / 32);
        __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(both[0] | both[1] << 8), s_rsrc, lane < 32 ? s_at : 0x80000000u,
                                              0, 0);
      } else {
        swap_bit<0xB1>(v[0], v[1], lane & 1);
        swap_bit<0xB1>(v[2], v[3], lane & 1);
        swap_bit<0x4E>(v[0], v[2], lane & 2);
        swap_bit<0x4E>(v[1], v[3], lane & 2);
#pragma unroll
        for (int t = 0; t < 4; ++t)
          __builtin_amdgcn_raw_buffer_store_b128(u32x4{v[t][0], v[t][1], v[t][2], v[t][3]}, rsrc,
                                                 base + (uint32_t)(32 * i + t) * row_bytes, 0, 2 /* nt */);
      }
    }
  }
  if constexpr (QUANT) {
    // the last column tile also writes the scale rows' padding behind it
    const uint32_t done = (uint32_t)((tc.n0 + C::OUTW) / 32);
    if (tc.n0 + C::OUTW >= g.N && done < s_bytes) {
      for (int r = tid; r < tc.rows_valid; r += C::THREADS)
        for (uint32_t z = done; z < s_bytes; z += 4)
          *reinterpret_cast<uint32_t*>(g.out_s + ((int64_t)tc.row0 + r) * s_bytes + z) = 0u;
    }
  }
}

template <class C, bool KTAIL, bool QUANT>
__global__ __launch_bounds__(C::THREADS) void mxfp4_pipe_kernel(MxGemmArgs g) {
  constexpr int BM = C::BM, BN = C::BN;
  constexpr int OPS = C::A_OPS + C::B_OPS;
  constexpr int TILE_N = C::OUTW;
  extern __shared__ __attribute__((aligned(1024))) unsigned char smem[];
  __shared__ MxProblems pl;

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  const int wave_u = __builtin_amdgcn_readfirstlane(wave);
  const int hh = lane >> 5;

  // prefix of the experts' row-tile counts, from the offsets clamped to the capacity (kept in the ring's memory until
  // the first loads)
  int2* first_offsets = reinterpret_cast<int2*>(smem);
  {
    constexpr int kPer = MOE_MAX_EXPERTS / C::THREADS;
    uint32_t mt[kPer], sum = 0;  // (unsigned: offsets that are no running sum can wrap the counts)
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      mt[i] = 0;
      if (e < g.E) {
        const int64_t lo = clamp_row(g.offsets[e], g.cap_rows), hi = clamp_row(g.offsets[e + 1], g.cap_rows);
        first_offsets[e] = int2{(int)lo, (int)hi};
        mt[i] = mx_row_tiles((int)lo, (int)hi, BM);
      }
      sum += mt[i];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const uint32_t up = __shfl_up(incl, off, 64);
      if (lane >= off) incl += up;
    }
    if (lane == 63) pl.wave_total[wave] = incl;
    __syncthreads();
    uint32_t run = incl - sum;
#pragma unroll
    for (int w = 0; w < C::NWAVES; ++w) run += w < wave ? pl.wave_total[w] : 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int e = tid * kPer + i;
      if (e <= g.E) pl.mt_prefix[e] = (int)run;
      run += mt[i];
    }
    if (tid == C::THREADS - 1 && g.E == MOE_MAX_EXPERTS) pl.mt_prefix[g.E] = (int)run;
    __syncthreads();
  }
  const int total_mt = pl.mt_prefix[g.E];
  const int n_tiles = (int)((g.N + TILE_N - 1) / TILE_N);
  // (tiles are counted in 31 bits: more have no memory to be stored in)
  const int64_t tiles64 = (int64_t)total_mt * n_tiles;
  const uint32_t total_tiles = (uint32_t)(tiles64 < 0 ? 0 : (tiles64 > 0x7FFFFFFF ? 0x7FFFFFFF : tiles64));
  const uint32_t t0 = (uint32_t)logical_worker();
  if (t0 >= total_tiles) return;
  const uint32_t my_tiles = (total_tiles - t0 + gridDim.x - 1) / gridDim.x;

  // Coordinates of this workgroup's tiles [from, from + kTableTiles), one a lane of the first wave.
  // Groups of kGroupRows row tiles sweep every column tile before the next group starts, so tiles that
  // run at the same time share rows and weights.
  auto fill_table = [&](uint32_t from, auto block_of) {
    if (tid < kTableTiles && from + tid < my_tiles) {
      const uint32_t t = t0 + (from + tid) * gridDim.x;
      const uint32_t span = (uint32_t)kGroupRows * (uint32_t)n_tiles, grp = t / span;
      const int in_group = (int)(t - grp * span);
      const int g0 = (int)grp * kGroupRows;
      const int gsize = total_mt - g0 < kGroupRows ? total_mt - g0 : kGroupRows;
      const int nt = in_group / gsize, gm = g0 + in_group - nt * gsize;
      int e = 0, hi_e = g.E;  // largest e with mt_prefix[e] <= gm
      while (hi_e - e > 1) {
        const int mid = (e + hi_e) >> 1;
        if (pl.mt_prefix[mid] <= gm) e = mid; else hi_e = mid;
      }
      const int2 block = block_of(e);
      const int64_t lo = block.x, hi = block.y;
      int64_t row0 = lo + ((int64_t)gm - pl.mt_prefix[e]) * BM;
      int64_t rows = hi - row0 < BM ? hi - row0 : BM;
      if (row0 < lo || row0 >= hi) row0 = rows = 0;  // wrapped counts
      pl.table[tid] = int4{e, (int)row0, (int)rows, nt * TILE_N};
    }
    __syncthreads();
  };
  auto coord = [&](uint32_t i) {
    const int4 v = pl.table[i % kTableTiles];
    return MxCoord{__builtin_amdgcn_readfirstlane(v.x), __builtin_amdgcn_readfirstlane(v.y),
                   __builtin_amdgcn_readfirstlane(v.z), __builtin_amdgcn_readfirstlane(v.w)};
  };
  fill_table(0, [&](int e) { return first_offsets[e]; });

  const int blocks = (int)mx_blocks(g.K);
  // stages: at least four, so that loads run at most one tile ahead (what lies past the row is zeros)
  const int nk = blocks <= 12 ? kRing : (blocks + 3) / 4;
  const uint32_t qp = (uint32_t)mx_row_bytes(g.K), sp = (uint32_t)mx_scale_bytes(g.K);
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  constexpr uint32_t kScaleBase = kRing * C::STAGE_BYTES;
  static_assert((kScaleBase & (kScaleBase - 1)) == 0, "ring offsets wrap with a mask");
  const bool gather = g.a_rows != nullptr;

  // The tile being loaded: each lane's 16-byte chunks as byte offsets from wave-uniform bases (the
  // host guarantees that they fit). Rows past the expert's block and columns past N point at valid
  // ones: they only feed outputs that are never stored. A wave load covers 16 rows of 4 chunks;
  // chunk c of row r is kept at position c ^ turn(r), which spreads 8 neighbouring rows over 128 bytes
  // of banks and 16 over 256. A lane's rows are 16 apart or more: one chunk for all.
  auto turn = [](int r) { return ((r >> 1) & 2) | (((r >> 1) ^ (r >> 3)) & 1); };
  const int chunk = (lane & 3) ^ turn(lane >> 2);
  uint64_t a_ptr, b_ptr, as_ptr, bs_ptr;  // of the next stage to load, and of the next group of scales
  int ik;                                 // that stage
  uint32_t scale_to = 0;                  // where in the scale ring that group goes
  uint32_t a_off[C::A_OPS], b_off[C::B_OPS], s_off[C::S_OPS];
  __amdgpu_buffer_rsrc_t a_rsrc, b_rsrc;
  int32_t slot_a[C::A_OPS], slot_s[C::S_OPS];  // gather: dispatch slots of the next tile's rows
  auto row_in = [&](const MxCoord& tc, int r) { return max(min(r, tc.rows_valid - 1), 0); };
  auto fetch_slots = [&](const MxCoord& tc) {
    const int32_t* rows = g.a_rows + tc.row0;
#pragma unroll
    for (int t2 = 0; t2 < C::A_OPS; ++t2) slot_a[t2] = rows[row_in(tc, 16 * (wave + C::NWAVES * t2) + (lane >> 2))];
#pragma unroll
    for (int t2 = 0; t2 < C::S_OPS; ++t2) {
      const int r = 64 * (wave_u + C::NWAVES * t2) + lane;
      slot_s[t2] = rows[row_in(tc, r < BM ? r : 0)];
    }
  };
  auto set_tile = [&](const MxCoord& tc) {
    const uint32_t last = (uint32_t)(g.a_tokens * g.a_k) - 1u;
    auto a_row = [&](int r, int32_t slot) -> uint32_t {
      if (!gather) return (uint32_t)row_in(tc, r);
      return (slot < 0 ? 0u : min((uint32_t)slot, last)) / (uint32_t)g.a_k;
    };
    auto b_row = [&](int r) -> uint32_t {
      const int half = C::GATED && r >= BN / 2 ? 1 : 0;
      int n = tc.n0 + (r - half * (BN / 2));
      if (n >= (int)g.N) n = tc.n0;
      return (uint32_t)(n + half * (int)g.N);
    };
    const int64_t a_first = gather ? 0 : tc.row0, b_first = (int64_t)tc.e * g.w_rows;
    a_ptr = uniform_addr(g.a_q + a_first * qp);
    b_ptr = uniform_addr(g.w_q + b_first * qp);
    as_ptr = uniform_addr(g.a_s + a_first * sp);
    ik = 0;
    bs_ptr = uniform_addr(g.w_s + b_first * sp);
#pragma unroll
    for (int t2 = 0; t2 < C::A_OPS; ++t2)
      a_off[t2] = a_row(16 * (wave + C::NWAVES * t2) + (lane >> 2), slot_a[t2]) * qp + chunk * 16;
#pragma unroll
    for (int t2 = 0; t2 < C::B_OPS; ++t2)
      b_off[t2] = b_row(16 * (wave + C::NWAVES * t2) + (lane >> 2)) * qp + chunk * 16;
#pragma unroll
    for (int t2 = 0; t2 < C::S_OPS; ++t2) {
      const int r = 64 * (wave_u + C::NWAVES * t2) + lane;
      s_off[t2] = (r < BM ? a_row(r, slot_s[t2]) : b_row(r - BM)) * sp;
    }
    if constexpr (KTAIL) {
      // (a tile without rows still reads row 0, and no row is shorter than the scalar offsets)
      const int64_t a_range = gather ? g.a_tokens * qp : (int64_t)max(tc.rows_valid, 1) * qp;
      a_rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(a_ptr), (short)0, (int)a_range, 0x00020000);
      b_rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(b_ptr), (short)0, (int)(g.w_rows * qp), 0x00020000);
    }
  };
  // Part `part` of `parts` of the loads of that stage into the ring at byte `to`; the first part of
  // a group's first stage also brings the group's scales, the last part moves on to the next stage.
  const uint32_t wave_lds = __builtin_amdgcn_readfirstlane(lds0 + (uint32_t)wave * 1024u);
  auto issue_part = [&](uint32_t to, int part, int parts) {
    const uint32_t sa = wave_lds + to, sb = sa + C::A_BYTES;
    if (part == 0 && (ik & (kGroup - 1)) == 0) {
#pragma unroll
      for (int t2 = 0; t2 < C::S_OPS; ++t2) {
        const int o = wave_u + C::NWAVES * t2;
        dma16_off(o * 64 < BM ? as_ptr : bs_ptr, s_off[t2], lds0 + kScaleBase + scale_to + (uint32_t)o * 1024u);
      }
      as_ptr += 16;
      bs_ptr += 16;
      scale_to = scale_to == 2 * C::SCALE_BYTES ? 0 : scale_to + C::SCALE_BYTES;
    }
    if constexpr (KTAIL) {
      // chunks past the row get an offset past the buffer resource's range and stage zeros; the scalar offset stays
      // inside the row also for the stages that a short one does not have
      const uint32_t soff = __builtin_amdgcn_readfirstlane(mx_stage_offset(ik, blocks));
      const bool in = chunk < blocks - 4 * ik;
#pragma unroll
      for (int t2 = 0; t2 < C::A_OPS; ++t2)
        if (t2 % parts == part)
          dma16_buf(a_rsrc, in ? a_off[t2] : 0x80000000u, soff, sa + (uint32_t)(C::NWAVES * t2 * 1024));
#pragma unroll
      for (int t2 = 0; t2 < C::B_OPS; ++t2)
        if ((C::A_OPS + t2) % parts == part)
          dma16_buf(b_rsrc, in ? b_off[t2] : 0x80000000u, soff, sb + (uint32_t)(C::NWAVES * t2 * 1024));
    } else {
#pragma unroll
      for (int t2 = 0; t2 < C::A_OPS; ++t2)
        if (t2 % parts == part) dma16_off(a_ptr, a_off[t2], sa + (uint32_t)(C::NWAVES * t2 * 1024));
#pragma unroll
      for (int t2 = 0; t2 < C::B_OPS; ++t2)
        if ((C::A_OPS + t2) % parts == part) dma16_off(b_ptr, b_off[t2], sb + (uint32_t)(C::NWAVES * t2 * 1024));
    }
    if (part == parts - 1) {
      ++ik;
      if constexpr (!KTAIL) {
        a_ptr += 64;
        b_ptr += 64;
      }
    }
  };

  f32x16 acc[C::FM][C::FN];
  u32x4 af[2][C::FM], bfr[2][C::FN];                         // fragments of a step: the one in use and the next
  uint32_t as[C::FM], bs[C::FN], as_next[C::FM], bs_next[C::FN];  // scale bytes of a stage, likewise (next: its words)
  // LDS addresses: the rows of a lane's fragments are multiples of 32 apart, so a lane needs one
  // address an operand (`turn` is the same for all), the rest are constant offsets.
  const int lrow = lane & 31;
  const int a_row0 = wm * C::WTM + lrow;
  const int b_row0 = wn * (C::GATED ? BN / 2 / C::WGN : C::WTN) + lrow;
  constexpr auto b_block = [](int j) { return C::GATED ? j / (C::FN / 2) * (BN / 2) + j % (C::FN / 2) * 32 : j * 32; };
  const uint32_t a_at = (uint32_t)(a_row0 * 64 + ((2 * hh) ^ turn(lrow)) * 16);
  const uint32_t b_at = (uint32_t)(C::A_BYTES + b_row0 * 64 + ((2 * hh) ^ turn(lrow)) * 16);
  const uint32_t as_at = kScaleBase + (uint32_t)(a_row0 * 16), bs_at = kScaleBase + (uint32_t)((BM + b_row0) * 16);
  auto load_frags = [&](int set, uint32_t at_byte, int ks) {
    const unsigned char* at = smem + ((a_at ^ (uint32_t)(ks * 16)) + at_byte);  // the step is the chunk's lowest bit
    const unsigned char* bt = smem + ((b_at ^ (uint32_t)(ks * 16)) + at_byte);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) af[set][i] = *reinterpret_cast<const u32x4*>(at + i * 32 * 64);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) bfr[set][j] = *reinterpret_cast<const u32x4*>(bt + b_block(j) * 64);
  };
  auto load_scales = [&](uint32_t at_byte) {
    const unsigned char* at = smem + (as_at + at_byte);
    const unsigned char* bt = smem + (bs_at + at_byte);
#pragma unroll
    for (int i = 0; i < C::FM; ++i) as_next[i] = *reinterpret_cast<const uint32_t*>(at + i * 32 * 16);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) bs_next[j] = *reinterpret_cast<const uint32_t*>(bt + b_block(j) * 16);
  };
  // The same reads for a next stage's first step, one at a time.
  auto read_next = [&](int q, uint32_t frag_byte, uint32_t scale_byte) {
    if (q < C::FM) af[0][q] = *reinterpret_cast<const u32x4*>(smem + (a_at + frag_byte) + q * 32 * 64);
    else if ((q -= C::FM) < C::FN) bfr[0][q] = *reinterpret_cast<const u32x4*>(smem + (b_at + frag_byte) + b_block(q) * 64);
    else if ((q -= C::FN) < C::FM) as_next[q] = *reinterpret_cast<const uint32_t*>(smem + (as_at + scale_byte) + q * 32 * 16);
    else if ((q -= C::FM) < C::FN) bs_next[q] = *reinterpret_cast<const uint32_t*>(smem + (bs_at + scale_byte) + b_block(q) * 16);
  };
  // This lane half's two bytes to the low half. Bytes past the row's last block may hold anything (255
  // is a NaN): their values are staged as zeros, so a scale of 2^-127 keeps them zero.
  auto take_scales = [&](int kt) {
    uint32_t keep = 0xFFFFu;
    if constexpr (KTAIL) {
      const int left = blocks - 4 * kt - 2 * hh;
      keep = left >= 2 ? keep : (left <= 0 ? 0u : 0xFFu);
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i) as[i] = KTAIL ? (as_next[i] >> (16 * hh)) & keep : as_next[i] >> (16 * hh);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) bs[j] = KTAIL ? (bs_next[j] >> (16 * hh)) & keep : bs_next[j] >> (16 * hh);
  };
  constexpr int kProducts = C::FM * C::FN, kReadsAll = 2 * (C::FM + C::FN);
  constexpr int kReads = kReadsAll > 2 * kProducts ? 3 : 2, kReadProducts = (kReadsAll + kReads - 1) / kReads;
  static_assert(kReadProducts <= kProducts && OPS <= kProducts, "the reads and the loads fit between the products");
  auto product = [&](int set, auto ks_c, int m) {
    constexpr int ks = decltype(ks_c)::value;
    const int j = m / C::FM, i = m % C::FM;
    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fp4_operand(bfr[set][j]), fp4_operand(af[set][i]),
                                                                acc[i][j], 4, 4, ks, (int)bs[j], ks, (int)as[i]);
  };
  constexpr std::integral_constant<int, 0> zero{};
  constexpr std::integral_constant<int, 1> one{};

  MxCoord tc = coord(0);
  if (gather) fetch_slots(tc);
  set_tile(tc);
#pragma unroll
  for (int q = 0; q < kRing; ++q) issue_part(q * C::STAGE_BYTES, 0, 1);
  wait_vmcnt_lds<3 * OPS, true>();  // the first stage and its scales
  bare_barrier();
  uint32_t ring = 0;      // where in the ring the stage being multiplied is
  uint32_t scale_at = 0;  // and its scales' words
  load_scales(0);
  load_frags(0, 0, 0);
  take_scales(0);
  for (uint32_t i_tile = 0;; ++i_tile) {
    const bool more = i_tile + 1 < my_tiles;
    MxCoord next = tc;  // behind the last tile its own first stages are loaded once more, for no use
    if (more) {
      if ((i_tile + 1) % kTableTiles == 0) {
        __syncthreads();  // every wave has read the last entry
        fill_table(i_tile + 1, [&](int e) {
          return int2{(int)clamp_row(g.offsets[e], g.cap_rows), (int)clamp_row(g.offsets[e + 1], g.cap_rows)};
        });
      }
      next = coord(i_tile + 1);
      if (gather) fetch_slots(next);
    }
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
    for (int kt = 0; kt < nk; ++kt) {
      load_frags(1, ring, 1);
#pragma unroll
      for (int m = 0; m < kProducts; ++m) product(0, zero, m);
      interleave_reads<kProducts, C::FM + C::FN>();
      // The second step's fragments are in registers before its products: the stage is handed over
      // first, so that they cover the barrier and the next fragments' latency. After the wait and
      // the barrier the next stage is complete for every wave and this one read by every wave: its
      // place takes the stage four on, loaded between the products (a wave waiting to issue a load
      // leaves the matrix unit to the other wave of its SIMD). Still under way may be the two stages
      // after the next, and for a tile's first three stages the previous tile's stores, issued behind
      // this tile's first four (before the first tile there are none).
      if (kt < 3 && i_tile != 0) wait_vmcnt_lds<2 * OPS + kTileStores<C, QUANT>, true>();
      else wait_vmcnt_lds<2 * OPS, true>();
      bare_barrier();
      const uint32_t to = ring;
      ring = (ring + C::STAGE_BYTES) & (kScaleBase - 1);
      // the row's next word of scales, or the next group's first (a tile starts one)
      const bool last = kt + 1 == nk;
      if (last || (kt & 3) == 3) scale_at = (scale_at & ~15u) == 2 * C::SCALE_BYTES ? 0 : (scale_at & ~15u) + C::SCALE_BYTES;
      else scale_at += 4;
      if (kt == nk - kRing) set_tile(next);
      // between the second step's products: first the next stage's LDS reads, then the loads
#pragma unroll
      for (int m = 0; m < kProducts; ++m) {
        product(1, one, m);
        __builtin_amdgcn_sched_barrier(0);
        if (m < kReadProducts) {
#pragma unroll
          for (int q = m * kReads; q < (m + 1) * kReads; ++q) read_next(q, ring, scale_at);
        }
        if (m >= kProducts - OPS) issue_part(to, m - (kProducts - OPS), OPS);
        __builtin_amdgcn_sched_barrier(0);
      }
      take_scales(last ? 0 : kt + 1);
    }
    store_tile<C, QUANT>(acc, g, tc);
    asm volatile("" : : : "memory");  // the stores stay here: the waits above count them
    if (!more) break;
    tc = next;
  }
  wait_vmcnt_lds<0, true>();  // no load may reach LDS after the workgroup has left it
}

template <class C, bool KTAIL, bool QUANT>
hipError_t launch_pipe(const MxGemmArgs& g, hipStream_t stream) {
  static std::atomic<bool> done[64] = {};
  auto kern = mxfp4_pipe_kernel<C, KTAIL, QUANT>;
  constexpr int lds = C::LDS_BYTES;
  const int dev = current_device();
  // Setting the attribute twice in a race of first calls is harmless.
  if (dev >= 0 && dev < 64 && !done[dev].load(std::memory_order_acquire)) {
    const hipError_t st = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                              hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (st != hipSuccess) return st;
    done[dev].store(true, std::memory_order_release);
  }
  static_assert(lds + sizeof(MxProblems) <= 160 * 1024, "the ring, the scales and the problem list fit in LDS");
  hipLaunchKernelGGL(kern, dim3(device_cu_count(dev)), dim3(C::THREADS), lds, stream, g);
  return hipGetLastError();
}

template <bool GATED>
using MxBig = std::conditional_t<GATED, MxTile<256, 256, 4, 2, true>, MxTile<256, 256, 2, 4, false>>;

template <bool GATED, bool QUANT = false>
hipError_t launch_products(const MxGemmArgs& g, hipStream_t stream) {
  if (g.cap_rows == 0) return hipSuccess;
  const int cus = device_cu_count(current_device());
  // The pipelined tiles address values and scales by 32-bit offsets: from the tile's first row (gathered: the first
  // token), and from one expert's weights. Below 2 GiB also where offset 2^31 marks a chunk past the row. What does not
  // fit takes the small tiles whatever its size, several times slower where there are many rows (532 and 108 us below).
  const int64_t qp = mx_row_bytes(g.K);
  const int64_t a_span = (g.a_rows != nullptr ? g.a_tokens : 256) * qp;
  const bool fits = a_span <= 0x7FFFFFFFll && g.w_rows * qp <= 0x7FFFFFFFll;
  // Small tiles while there are few of them: a call of small tiles takes 5 us and up, one of pipelined tiles 10, but a
  // pipelined tile does 16 times the work in 2 to 4 times a small one's time. (The host knows the capacity, not the
  // spread: half a tile more per expert.) The limit is 3 + 3000 / (K + 256) a CU; small and pipelined, plain products:
  // 1012 rows of 6 experts 240 -> 32 5.3 and 10.2 us; 4091 rows of 8 experts 392 -> 520 (1188 small tiles) 9.6 and 13.6;
  // 3706 rows of 81 experts 120 -> 976 (2480) 13.2 and 16.9; 4284 rows of 3 experts 392 -> 1432 (3082) 19 and 17; 864
  // rows of 11 experts 1528 -> 2480 (1248) 27 and 20; 65536 rows of 64 experts 768 -> 2048 532 and 108. And below a mean
  // of 32 rows per expert, where pipelined tiles are mostly empty: gate/up of 64 experts 2048 -> 2 x 768, evenly spread /
  // skewed, 16 rows 30 and 42 / 36 and 42 us, 32 rows 35 and 42 / 45 and 43, 64 rows 60 and 44 / 70 and 45. Over 430
  // calls of random sizes the choice costs 0.2% against the better of the two (always small 8%, always pipelined 78%).
  const int64_t used = g.cap_rows < g.E ? g.cap_rows : g.E;
  const int64_t small_tiles = (g.cap_rows / 32 + used / 2) * ((g.N + kThinCols<GATED> - 1) / kThinCols<GATED>);
  const bool small = small_tiles * (g.K + 256) <= cus * (3 * (g.K + 256) + 3000) || g.cap_rows < (int64_t)32 * g.E;
  if (fits && !small) {
    if (g.K % kStageK != 0 || g.K < kRing * kStageK) return launch_pipe<MxBig<GATED>, true, QUANT>(g, stream);
    return launch_pipe<MxBig<GATED>, false, QUANT>(g, stream);
  }
  hipLaunchKernelGGL((mxfp4_thin_kernel<GATED, QUANT, 2>), dim3(cus * 4), dim3(kThinThreads), 0, stream, g);
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
                                       int64_t cap_rows, int64_t d, int64_t h, int32_t E, uint16_t* h_buf, uint8_t* h_q,
                                       uint8_t* h_s, hipStream_t stream) {
  const MxGemmArgs g{x_q, x_s, perm, k, x_rows, w_q, w_s, 2 * h, h, d, offsets, E, cap_rows, h_buf, h, h_q, h_s};
  return h_buf != nullptr ? launch_products<true>(g, stream) : launch_products<true, true>(g, stream);
}

}  // namespace moe
