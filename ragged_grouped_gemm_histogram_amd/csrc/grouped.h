// Device pieces shared by the grouped GEMM kernels: tile geometry, the problem list built from the
// device offsets, direct global -> LDS loads, waits and barriers, and the epilogue. A stage holds
// 128 bytes of every tile row (8 chunks of 16 bytes), whatever the operands' type.
#pragma once

#include "common.h"

namespace moe {

constexpr int BK = 64;         // K per stage: 8 chunks of 16 bytes per tile row
constexpr int kChunksK = BK / 8;
constexpr int kGroupM = 8;     // m-tiles per group in the tile order (operand reuse in L2)

// Tile geometry: BM x BN weight rows per workgroup, WGM x WGN waves, NST LDS stages.
template <int BM_, int BN_, int WGM_, int WGN_, int NST_, bool GATED_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, NST = NST_;
  static constexpr bool GATED = GATED_;
  static constexpr int NWAVES = WGM * WGN, THREADS = 64 * NWAVES;
  static constexpr int WTM = BM / WGM, WTN = BN / WGN;  // wave tile
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int OUTW = GATED ? BN / 2 : BN;  // output columns per tile
  static constexpr int OUT_CPR = OUTW / 8;          // 16-byte chunks per output row
  static constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
  static constexpr int LDS_BYTES = NST * STAGE_BYTES;
  static constexpr int A_LOADS = BM * kChunksK / THREADS;  // register path: 16-byte chunks per thread
  static constexpr int B_LOADS = BN * kChunksK / THREADS;
  static constexpr int A_OPS = A_BYTES / 1024 / NWAVES;  // pipelined path: 1 KB wave loads per wave per stage
  static constexpr int B_OPS = B_BYTES / 1024 / NWAVES;
  static_assert(WTM % 32 == 0 && WTN % 32 == 0, "wave tile must split into 32x32 blocks");
  static_assert(BM * OUTW * 2 <= LDS_BYTES, "epilogue tile must fit in the stage buffers");
  static_assert((OUT_CPR & (OUT_CPR - 1)) == 0, "output chunk count must be a power of two");
  static_assert(!GATED || FN % 2 == 0, "gated tiles pair gate and up blocks");
  static_assert(A_BYTES % (1024 * NWAVES) == 0 && B_BYTES % (1024 * NWAVES) == 0, "stage must split into wave loads");
};

template <int THREADS>
struct ProblemList {
  int seg_lo[MOE_MAX_EXPERTS];
  int seg_rows[MOE_MAX_EXPERTS];
  int mt_prefix[MOE_MAX_EXPERTS + 1];
  int scan_tmp[THREADS / 64];  // one total per wave
};

struct TileCoord {
  int e;
  int mi;
  int64_t row0;     // first sorted row of the tile
  int rows_valid;   // rows of the tile inside the expert's block
  int64_t n0;       // first output column
};

// K-contiguous tile rows are 128 B (8 chunks of 16 B). LDS has 64 banks (256 B
// per cycle), so two rows share a bank window and a 16-lane read group spans 16
// rows: chunk c of row r is kept at position c ^ ((r / 2) % 8), which gives the
// 16 rows of a group 16 distinct (window half, position) pairs.
__device__ __forceinline__ int swz(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// N-contiguous rows (W_down tiles) are BN*2 bytes. A 32-lane half of a transpose
// read touches 4 rows x 4 consecutive chunks; chunk c of row k is kept at
// c ^ (4 * (k % 4)), which spreads those 16 chunks over the 16 bank positions.
__device__ __forceinline__ int swz_n(int krow, int chunk) { return chunk ^ (4 * (krow & 3)); }

// One 16-byte chunk per lane from base + off (bytes) into LDS[lds_addr + 16 * lane]: a
// wave-uniform 64-bit base in SGPRs and a per-lane 32-bit byte offset (M0 holds the
// wave's LDS base).
__device__ __forceinline__ void dma16_off(uint64_t base, uint32_t off, uint32_t lds_addr) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :
               : "v"(off), "s"(base), "s"(lds_addr)
               : "memory", "m0");
}

// One 16-byte chunk per lane through a buffer resource into LDS[lds_addr + 16 * lane]: a lane whose
// offset lies past the resource's range reads nothing and stages zeros.
__device__ __forceinline__ void dma16_buf(__amdgpu_buffer_rsrc_t rsrc, uint32_t off, uint32_t soff, uint32_t lds_addr) {
  lds_addr = __builtin_amdgcn_readfirstlane(lds_addr);  // the same in every lane: M0 takes it from an SGPR
  asm volatile("s_mov_b32 m0, %3\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               :
               : "v"(off), "s"(rsrc), "s"(soff), "s"(lds_addr)
               : "memory", "m0");
}

// A 64-bit value every lane holds the same value of, moved to SGPRs.
__device__ __forceinline__ int64_t uniform_i64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)v >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// A pointer every lane holds the same value of, moved to SGPRs.
__device__ __forceinline__ uint64_t uniform_addr(const void* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | lo;
}

// vmcnt(N) together with lgkmcnt(0): this wave's own LDS reads are complete
// too, whatever order the compiler left them in, before a barrier after which
// other waves may overwrite the slot those reads came from.
//
// EXACT: issue it as the compiler's own s_waitcnt, so that its wait bookkeeping knows every
// earlier LDS read is complete and adds no wait of its own for them behind newer reads.
// s_waitcnt's immediate on gfx9: vmcnt in bits [3:0] and [15:14], expcnt in [6:4] (7: no
// wait), lgkmcnt in [11:8].
template <int N, bool EXACT = false>
__device__ __forceinline__ void wait_vmcnt_lds() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  if constexpr (EXACT) __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ void bare_barrier() { asm volatile("s_barrier" : : : "memory"); }

// Barrier for LDS hand-offs only: this wave's LDS accesses are complete, its
// global stores may still be in flight (a full __syncthreads would wait for
// their write acknowledgements too).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" : : : "memory"); }

// Scheduling hint for one K slice: spread READS LDS reads (the next slice's
// fragments) between the MFMAS matrix instructions of the current one, so the
// reads' latency hides behind matrix work instead of stalling the next slice.
template <int MFMAS, int READS>
__device__ __forceinline__ void interleave_reads() {
  constexpr int kPer = MFMAS / READS > 0 ? MFMAS / READS : 1;
  constexpr int kPairs = READS < MFMAS ? READS : MFMAS;
#pragma unroll
  for (int i = 0; i < kPairs; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);  // MFMA
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // LDS read
  }
  if constexpr (MFMAS > kPairs * kPer) __builtin_amdgcn_sched_group_barrier(0x008, MFMAS - kPairs * kPer, 0);
  if constexpr (READS > kPairs) __builtin_amdgcn_sched_group_barrier(0x100, READS - kPairs, 0);
}

// Map a persistent workgroup to a logical worker so that consecutive logical
// workers (which take consecutive tiles) sit on one XCD: workgroups are
// dealt to the 8 XCDs round-robin.
__device__ __forceinline__ int logical_worker() {
  const int G = gridDim.x, b = blockIdx.x;
  if (G % 8 != 0) return b;
  return (b % 8) * (G / 8) + b / 8;
}

// Problem list from the device offsets, clamped so no access leaves the buffers:
// per expert its first row, its row count and the prefix of its m-tile counts.
template <int BM, int THREADS, class Args>
__device__ void build_problem_list(const Args& g, ProblemList<THREADS>& pl) {
  const int tid = threadIdx.x;
  constexpr int kPer = (MOE_MAX_EXPERTS + THREADS - 1) / THREADS;
  int mt_local[kPer];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    int mt = 0;
    if (e < g.E) {
      int64_t lo = g.offsets[e], hi = g.offsets[e + 1];
      lo = lo < 0 ? 0 : (lo > g.cap_rows ? g.cap_rows : lo);
      hi = hi < lo ? lo : (hi > g.cap_rows ? g.cap_rows : hi);
      pl.seg_lo[e] = (int)lo;
      pl.seg_rows[e] = (int)(hi - lo);
      mt = (int)((hi - lo + BM - 1) / BM);
    }
    mt_local[i] = mt;
    sum += mt;
  }
  // Exclusive prefix of the per-thread sums: an inclusive scan inside each wave (shuffles), the
  // waves' totals through LDS, then each thread adds the totals of the waves before it.
  constexpr int kWaves = THREADS / 64;
  const int lane = tid & 63, wave = tid >> 6;
  int incl = sum;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int up = __shfl_up(incl, off, 64);
    if (lane >= off) incl += up;
  }
  if (lane == 63) pl.scan_tmp[wave] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int v = pl.scan_tmp[w];
    before += w < wave ? v : 0;
    total += v;
  }
  int run = before + incl - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int e = tid * kPer + i;
    if (e < g.E) pl.mt_prefix[e] = run;
    run += mt_local[i];
  }
  if (tid == 0) pl.mt_prefix[g.E] = total;
  __syncthreads();
}

// Tile t -> (expert, m-tile, n-tile). Groups of GM consecutive m-tiles
// sweep every n-tile before the next group starts, so tiles that run at the
// same time share A rows and weight rows.
template <int BM, int TILE_N, int THREADS>
__device__ __forceinline__ TileCoord tile_coord(int64_t t, int64_t n_tiles, int total_mt, int E,
                                                const ProblemList<THREADS>& pl, int group_m = kGroupM) {
  const int kGroupM = group_m;
  const int64_t group_span = (int64_t)kGroupM * n_tiles;
  const int64_t group = t / group_span;
  const int64_t in_group = t - group * group_span;
  const int64_t g0 = group * kGroupM;
  const int gsize = (int)((total_mt - g0) < kGroupM ? (total_mt - g0) : kGroupM);
  const int64_t nt = in_group / gsize;
  const int gm = (int)(g0 + (in_group - nt * gsize));
  int lo_e = 0, hi_e = E;  // largest e with mt_prefix[e] <= gm: the non-empty expert owning m-tile gm
  while (hi_e - lo_e > 1) {
    const int mid = (lo_e + hi_e) >> 1;
    if (pl.mt_prefix[mid] <= gm) lo_e = mid; else hi_e = mid;
  }
  // every lane holds the same coordinates (LDS reads of the problem list): keep them in scalar
  // registers, where the epilogue's buffer descriptor and the load bases need them
  TileCoord c;
  c.e = __builtin_amdgcn_readfirstlane(lo_e);
  c.mi = __builtin_amdgcn_readfirstlane(gm - pl.mt_prefix[lo_e]);
  c.row0 = uniform_i64((int64_t)pl.seg_lo[lo_e] + (int64_t)c.mi * BM);
  c.rows_valid = __builtin_amdgcn_readfirstlane(min(BM, pl.seg_rows[lo_e] - c.mi * BM));
  c.n0 = uniform_i64(nt * TILE_N);
  return c;
}

// weight-tile row of a wave's fn-th 32-row block (gated: the first FN/2 blocks are gate rows,
// the rest the matching up rows, BN/2 further down)
template <class C>
__device__ __forceinline__ int b_block_row(int wn, int fn) {
  if constexpr (C::GATED) {
    constexpr int half_fn = C::FN / 2;
    const int half = fn / half_fn, sub = fn % half_fn;
    return half * (C::BN / 2) + wn * (C::BN / 2 / C::WGN) + sub * 32;
  } else {
    return wn * C::WTN + fn * 32;
  }
}

// SiLU(g) * u in fp32 with the hardware
// exponential and reciprocal (a few fp32 ulps, far below the bf16 rounding of the result).
__device__ __forceinline__ float swiglu(float gv, float uv) { return gv * __builtin_amdgcn_rcpf(1.0f + __expf(-gv)) * uv; }

// threadIdx.x, through an opaque register move when OPAQUE: the epilogues' LDS and global
// addresses are fixed per lane, so the compiler otherwise computes them once before the tile
// loop and keeps them (about 60 registers) live through every main loop. The 256-row tiles with
// a plain (256-column) output need those registers for the second fragment set, and the
// U-keeping and weight-gradient launches to avoid spilling; the other tiles are faster with the
// addresses kept.
template <bool OPAQUE>
__device__ __forceinline__ int epilogue_tid() {
  int tid = threadIdx.x;
  if constexpr (OPAQUE) asm volatile("" : "+v"(tid));
  return tid;
}
template <class C>
constexpr bool kOpaqueEpilogue = !C::GATED && C::BM == 256;

// Registers -> bf16 tile in LDS (swizzled 16-byte chunks) -> global. For the
// gated projection, SwiGLU is applied here: g and u are rounded to bf16 first,
// then SiLU(g) * u is evaluated in fp32 with the hardware exponential and
// reciprocal (a few fp32 ulps, far below the bf16 rounding of the result).
// acc[i][j][4q+s] is output row (wm*WTM + i*32 + lane%32), column
// (block column base + 8q + 4*(lane/32) + s).
template <class C, class Args>
__device__ __forceinline__ void epilogue(const f32x16 (&acc)[C::FM][C::FN], unsigned char* smem, const Args& g,
                                         const TileCoord& tc) {
  constexpr int BM = C::BM, BN = C::BN;
  const int tid = epilogue_tid<kOpaqueEpilogue<C>>(), lane = tid & 63, wave = tid >> 6;
  const int wm = wave / C::WGN, wn = wave % C::WGN;
  unsigned char* ot = smem;  // [BM][OUTW] bf16
  constexpr int OUT_ROW_BYTES = C::OUTW * 2;
  const int half_lane = lane >> 5;
  if constexpr (C::GATED) {
    constexpr int half_fn = C::FN / 2;
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int r = wm * C::WTM + i * 32 + (lane & 31);
#pragma unroll
      for (int j = 0; j < half_fn; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float hv[4];
          // g and u rounded to bf16 two at a time (one packed convert per pair)
#pragma unroll
          for (int s = 0; s < 4; s += 2) {
            const uint32_t g2 = pack_bf16x2(acc[i][j][4 * q + s], acc[i][j][4 * q + s + 1]);
            const uint32_t u2 = pack_bf16x2(acc[i][j + half_fn][4 * q + s], acc[i][j + half_fn][4 * q + s + 1]);
            hv[s] = swiglu(bf16_bits_to_f32(g2 & 0xFFFFu), bf16_bits_to_f32(u2 & 0xFFFFu));
            hv[s + 1] = swiglu(bf16_bits_to_f32(g2 >> 16), bf16_bits_to_f32(u2 >> 16));
          }
          const int col = wn * (BN / 2 / C::WGN) + j * 32 + 8 * q + 4 * half_lane;
          const int c = col >> 3;
          uint2 pk{pack_bf16x2(hv[0], hv[1]), pack_bf16x2(hv[2], hv[3])};
          *reinterpret_cast<uint2*>(ot + r * OUT_ROW_BYTES + ((c ^ (r & (C::OUT_CPR - 1))) * 16) + (col & 7) * 2) = pk;
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) {
      const int r = wm * C::WTM + i * 32 + (lane & 31);
#pragma unroll
      for (int j = 0; j < C::FN; ++j) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int col = wn * C::WTN + j * 32 + 8 * q + 4 * half_lane;
          const int c = col >> 3;
          uint2 pk{pack_bf16x2(acc[i][j][4 * q + 0], acc[i][j][4 * q + 1]),
                   pack_bf16x2(acc[i][j][4 * q + 2], acc[i][j][4 * q + 3])};
          *reinterpret_cast<uint2*>(ot + r * OUT_ROW_BYTES + ((c ^ (r & (C::OUT_CPR - 1))) * 16) + (col & 7) * 2) = pk;
        }
      }
    }
  }
  lds_barrier();
  // Thread tid takes chunk tid % OUT_CPR of rows tid / OUT_CPR + RSTEP * it: all its LDS reads
  // first, then the stores (one read's latency instead of one per store). The stores go through a
  // buffer resource that ends at the tile's last valid row, and a column past N gets an offset
  // past the end: the hardware drops those stores, so no branch separates them.
  constexpr int kStoreIters = BM * C::OUT_CPR / C::THREADS;
  constexpr int RSTEP = C::THREADS / C::OUT_CPR;
  static_assert(C::THREADS % C::OUT_CPR == 0, "a thread keeps one chunk column");
  const int c = tid % C::OUT_CPR, r0 = tid / C::OUT_CPR;
  u32x4 v[kStoreIters];
#pragma unroll
  for (int it = 0; it < kStoreIters; ++it) {
    const int r = r0 + RSTEP * it;
    v[it] = *reinterpret_cast<const u32x4*>(ot + r * OUT_ROW_BYTES + ((c ^ (r & (C::OUT_CPR - 1))) * 16));
  }
  const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
      g.out + tc.row0 * g.ldo, (short)0, (int)((int64_t)tc.rows_valid * g.ldo * 2), 0x00020000);
  const int64_t col = tc.n0 + c * 8;
  const uint32_t col_off = col < g.N ? (uint32_t)(col * 2) : 0x80000000u;
  const uint32_t row_bytes = (uint32_t)(g.ldo * 2);
#pragma unroll
  for (int it = 0; it < kStoreIters; ++it) {
    const uint32_t off = (uint32_t)(r0 + RSTEP * it) * row_bytes + col_off;
    // Plain outputs (the down projection's y_perm, 256-column tiles) go out as non-temporal
    // stores: this launch never reads them back, and allocating them in L2 would evict operand
    // lines (-2% on the down projection in the zipf64 step, -8% back to back).
    __builtin_amdgcn_raw_buffer_store_b128(v[it], rsrc, off, 0, C::GATED ? 0 : 2 /* nt */);
  }
  lds_barrier();  // LDS is reused by the next tile
}

}  // namespace moe
