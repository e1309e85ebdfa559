// Norms around a block on the residual stream, forward and backward. For a row r of the stream and the
// block's output y, with rs(x) = 1 / sqrt(mean x^2 + eps):
//
//   u  = y rs(y) w_post     (or y)              r' = a r + b gate u          n = r' rs(r') w_next
//
// Backward, with x = r', h = dn w_next, k1 = rs(x), k2 = k1^3 mean(h x):
//
//   g = dr' + k1 h - k2 x      dr = a g      dw_next = sum_t dn x k1      du = b gate g
//   dgate = b sum g u          dw_post = sum_t du y rs(y)
//   dy = rs(y) du w_post - rs(y)^3 mean(du w_post y) y      (or du)
//
// Both are bound by HBM: each input is read once, into registers, and each output written once. All
// sums over a row come of one round: sum q g with q = gate w_post y is D + k1 E - k2 F for the sums D, E,
// F of q dr', q h and q x, so nothing of the second norm waits for the first, and no statistics of the
// forward are kept. Everything is fp32 after the loads; each output is rounded once.
//
// A row belongs to a team of ceil(d / 512) waves (half as many above 8192), a lane holding 8
// consecutive columns (twice 8); up to 256 columns a wave takes two rows at once, up to 128 four. The
// backward's teams walk the rows with the column sums in registers; a workgroup joins its teams' and leaves
// one row of partial sums, which a second launch adds in order, so results repeat bit for bit.
//
// Measured (bf16 / fp32 stream; a copy of 2 GiB runs at 4.9 TB/s, tensors that the last-level cache holds run faster):
//                                 before              after, both norms   backward of each
//   65536 x 64                    7.8 / 7.5 us        9.7 / 12.1          15.2 / 16.0, 22.4 / 23.4
//   8191 x 2880                   16.5 / 22.8         30.5 / 55.4         36.1 / 64.4, 60.4 / 93.5
//   4096 x 8192                   21.3 / 30.7         41.9 / 78.6         50.0 / 90.5, 99.7 / 136.7
//   2048 x 16384                  21.3 / 31.7         51.4 / 87.2         55.1 / 98.8, 156 / 218
// The last column's last row is 2.6 to 2.8 TB/s: above 8192 columns a lane's two vectors of all rows and sums leave no
// registers to read ahead. Backwards with both norms spill there, with a gate per channel 46 registers (bf16) and 65 (fp32;
// 53 and 90 with a second part of dn), without one 4 and 26; from 4097 columns on 18 and 34 (26 and 44), and none and 4; with
// an fp32 stream and narrower rows one. Small calls wait for one chain of load, sum and store, 3 us, and the backward's second launch.

#include "common.h"
#include "norm.h"

namespace moe {
namespace {

constexpr int kMaxWaves = 16;

struct NormArgs {
  const void* r;         // stream: forward before the block, backward r'
  const uint16_t* y;
  const void* w_post;    // NULL: ones
  const void* w_next;
  const void* gate;      // per token fp32, per channel as the weights
  int gate_kind;
  bool w_f32;
  float a, b, eps;
  int64_t T;
  int d;
  void* r_out;           // backward: dr
  uint16_t* n_out;
  const void* dr;        // backward only
  const uint16_t* dn;
  const uint16_t* dn_add;  // a second part of it, or NULL
  uint16_t* dy;
  float* d_gate_token;
  float* partial;        // [workgroups][sums][d]
  int team_waves;
};

typedef float f32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  const u32x4 x = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_bits_to_f32(x[i] & 0xFFFFu);
    v[2 * i + 1] = __builtin_bit_cast(float, x[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4_t x = reinterpret_cast<const f32x4_t*>(p)[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[4 * i + j] = x[j];
  }
}

__device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<u32x4*>(p) = o;
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4_t o = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    reinterpret_cast<f32x4_t*>(p)[i] = o;
  }
}

// Columns of a weight (ones where there is none).
__device__ __forceinline__ void load_weight(const void* w, bool f32, int col, float (&v)[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
  } else if (f32) {
    load8(static_cast<const float*>(w) + col, v);
  } else {
    load8(static_cast<const uint16_t*>(w) + col, v);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  const int y = __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, x), CTRL, 0xF, 0xF, true);
  return x + __builtin_bit_cast(float, y);
}

// Sum over each row of 16 lanes, the same in every lane.
__device__ __forceinline__ float sum16(float x) {
  x = dpp_add<0xB1>(x);          // neighbours
  x = dpp_add<0x4E>(x);          // pairs
  x = dpp_add<0x141>(x);         // quads of a half row
  return dpp_add<0x140>(x);      // halves
}

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

__device__ __forceinline__ float wave_sum(float x) {
  x = sum16(x);
  return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}

// x of this row of 16 lanes and of the one beside it, added up; and of both halves of the wave.
__device__ __forceinline__ float add_rows(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
__device__ __forceinline__ float add_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}

// Sums over a team of `waves` waves from wave `first` of the workgroup on, the same in every lane; with LANES below 64
// over the LANES lanes that hold a row. `buf` alternates between two LDS areas, so one barrier a round is enough: a wave
// reaches the round after next only behind the next one's barrier.
template <int LANES, int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*red)[kMaxWaves][N], int& buf, int waves, int first = 0) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = LANES == 64 ? wave_sum(v[i]) : (LANES == 32 ? add_rows(sum16(v[i])) : sum16(v[i]));
  if (LANES < 64 || waves == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[buf][wave][i] = v[i];
  }
  __syncthreads();
  const int from = lane & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = sum16(from < waves ? red[buf][first + from][i] : 0.0f);
  buf ^= 1;
}

// LANES: lanes that hold a row, 64 for a team of waves; with fewer a wave takes several rows.
template <class S, bool BRANCH, bool POST, bool NEXT, int V, int LANES>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_kernel(NormArgs g) {
  __shared__ float red[2][kMaxWaves][1];
  const int waves = blockDim.x >> 6;
  const S* r_in = static_cast<const S*>(g.r);
  S* r_out = static_cast<S*>(g.r_out);
  const float inv_d = 1.0f / (float)g.d;
  int buf = 0;
  constexpr int kRows = 64 / LANES;
  const int lane = threadIdx.x & 63;
  const int span = LANES == 64 ? (int)blockDim.x : LANES, at = LANES == 64 ? (int)threadIdx.x : lane % LANES;
  const int64_t turn = LANES == 64 ? gridDim.x : (int64_t)gridDim.x * waves * kRows;
  for (int64_t t0 = LANES == 64 ? blockIdx.x : ((int64_t)blockIdx.x * waves + (threadIdx.x >> 6)) * kRows; t0 < g.T; t0 += turn) {
    const int64_t t = LANES == 64 ? t0 : t0 + lane / LANES;
    const int64_t row = t * g.d;
    const int end = LANES == 64 || t < g.T ? g.d : 0;  // columns of this lane's row
    float x[V][8], u[V][8];
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * span + at) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = u[j][i] = 0.0f;
      if (col < end) {
        load8(r_in + row + col, x[j]);
        if constexpr (BRANCH) load8(g.y + row + col, u[j]);
      }
    }
    if constexpr (BRANCH) {
      float scale = g.b;
      if (g.gate_kind == MOE_GATE_TOKEN && end > 0) scale *= static_cast<const float*>(g.gate)[t];
      if constexpr (POST) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[0] = fmaf(u[j][i], u[j][i], ss[0]);
        team_sum<LANES>(ss, red, buf, waves);
        scale *= rsqrtf(fmaf(ss[0], inv_d, g.eps));
        ss[0] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * span + at) * 8;
        if (col < end) {
          float w[8];
          if constexpr (POST) {
            load_weight(g.w_post, g.w_f32, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[j][i] *= w[i];
          }
          if (g.gate_kind == MOE_GATE_CHANNEL) {
            load_weight(g.gate, g.w_f32, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) u[j][i] *= w[i];
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] = fmaf(g.a, x[j][i], scale * u[j][i]);
          store8(r_out + row + col, x[j]);
        }
      }
    }
    if constexpr (NEXT) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(x[j][i], x[j][i], ss[0]);
      team_sum<LANES>(ss, red, buf, waves);
      const float rs = rsqrtf(fmaf(ss[0], inv_d, g.eps));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * span + at) * 8;
        if (col < end) {
          float w[8];
          load_weight(g.w_next, g.w_f32, col, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] *= x[j][i] * rs;
          store8(g.n_out + row + col, w);
        }
      }
    }
  }
}

// A row of a tensor as a buffer resource: what lies behind its `bytes` reads as zeros and is not written, so lanes
// past the last column, rows past the last and tensors that are not there need no branches.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_of(const void* base, int64_t offset, int bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base) + (uint64_t)offset;
  // (readfirstlane gives an int: its sign must not reach the upper half)
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)at), hi = __builtin_amdgcn_readfirstlane((uint32_t)(at >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)hi << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

__device__ __forceinline__ u32x4 read16(__amdgpu_buffer_rsrc_t row, uint32_t at) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(row, at, 0, 0));
}

// Eight columns as they are read, from column `col` of a row on.
template <class S>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4 v;
  __device__ __forceinline__ void read(__amdgpu_buffer_rsrc_t row, int col) { v = read16(row, col * 2); }
  __device__ __forceinline__ void keep() { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ float operator[](int i) const {
    return __builtin_bit_cast(float, i & 1 ? v[i >> 1] & 0xFFFF0000u : v[i >> 1] << 16);
  }
};
template <>
struct Raw<float> {
  u32x4 lo, hi;
  __device__ __forceinline__ void read(__amdgpu_buffer_rsrc_t row, int col) {
    lo = read16(row, col * 4), hi = read16(row, col * 4 + 16);
  }
  __device__ __forceinline__ void keep() { asm volatile("" : "+v"(lo), "+v"(hi)); }
  __device__ __forceinline__ float operator[](int i) const { return __builtin_bit_cast(float, i < 4 ? lo[i] : hi[i - 4]); }
};

__device__ __forceinline__ void write8(__amdgpu_buffer_rsrc_t row, int col, const float (&v)[8], uint16_t) {
  u32x4 o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  __builtin_amdgcn_raw_buffer_store_b128(o, row, col * 2, 0, 0);
}
__device__ __forceinline__ void write8(__amdgpu_buffer_rsrc_t row, int col, const float (&v)[8], float) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4_t o = {v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o), row, col * 4 + 16 * i, 0, 0);
  }
}

// One row of the backward's inputs, a lane's columns of it.
template <class S, int V>
struct BackRow {
  Raw<S> x[V], d[V];
  Raw<uint16_t> dn[V], more[V], y[V];
  float gate;  // one per token
};

constexpr int kBackWaves = 8;  // a workgroup: as many teams as fit, one WIDE team above
// For the weights, their columns rounded up to 512 a wave (1024 with V = 2): three up to 10240 columns, two up to 16384.
constexpr int kBackLds = 128 * 1024;

// CHANNEL: the gate is one per channel. ADD: d_n comes in two parts. The column sums stand in the order dw_next,
// dw_post, dgate, those that the form has. A row's loads go out before the row before it is computed (not with V = 2, nor
// with several rows a wave, whose registers do not hold two turns); for that the weights come from LDS: loads return
// in order, so one of a weight would wait for the whole row read ahead. WIDE: a team of more than 8 waves. LANES as above.
template <class S, bool BRANCH, bool POST, bool NEXT, bool CHANNEL, bool ADD, bool WIDE, int V, int LANES>
__global__ __launch_bounds__(64 * (WIDE ? kMaxWaves : kBackWaves), 4) void norm_backward_kernel(NormArgs g) {
  constexpr int kCols = (NEXT ? 1 : 0) + (POST ? 1 : 0) + (CHANNEL ? 1 : 0);
  constexpr int kColPost = NEXT ? 1 : 0, kColGate = kColPost + (POST ? 1 : 0);
  __shared__ float red[2][kMaxWaves][6];
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  float* w_lds = reinterpret_cast<float*>(lds);  // the weights in the order of their sums as fp32, 0 past the last column
  constexpr int kRows = 64 / LANES;  // rows of a team's turn
  const int waves = g.team_waves, span = LANES == 64 ? 64 * waves : LANES, padded = span * 8 * V;
  const int team = __builtin_amdgcn_readfirstlane(((int)threadIdx.x >> 6) / waves);  // (divided in vector registers: rows and addresses of rows shall be scalar)
  const int at = LANES == 64 ? (int)threadIdx.x - team * span : (int)threadIdx.x & (LANES - 1);
  const int sub = LANES == 64 ? 0 : ((int)threadIdx.x & 63) / LANES;  // this lane's row of the turn
  const float inv_d = 1.0f / (float)g.d;
  const bool token = BRANCH && g.gate_kind == MOE_GATE_TOKEN;
  const bool in_lds = !WIDE || kCols * padded * (int)sizeof(float) <= kBackLds;
  const int s_bytes = g.d * (int)sizeof(S), h_bytes = g.d * 2;  // a row of the stream, of the block's side
  const void* sources[3] = {nullptr, nullptr, nullptr};
  if constexpr (NEXT) sources[0] = g.w_next;
  if constexpr (POST) sources[kColPost] = g.w_post;
  if constexpr (CHANNEL) sources[kColGate] = g.gate;
  auto load_padded = [&](int k, int col, float (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 0.0f;
    if (col < g.d) load_weight(sources[k], g.w_f32, col, w);
  };
  if (in_lds) {
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      for (int col = threadIdx.x * 8; col < padded; col += blockDim.x * 8) {
        float w[8];
        load_padded(k, col, w);
        store8(w_lds + k * padded + col, w);
      }
    __syncthreads();
  }
  auto weight = [&](int k, int col, float (&w)[8]) {
    if (in_lds) load8(w_lds + k * padded + col, w);
    else load_padded(k, col, w);
  };
  float acc[kCols > 0 ? kCols : 1][V][8];
#pragma unroll
  for (int k = 0; k < kCols; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][j][i] = 0.0f;

  // rows from t on that are there
  auto rows_at = [&](int64_t t) { return t >= g.T ? 0 : (g.T - t < kRows ? (int)(g.T - t) : kRows); };
  // where a column stands behind the turn's first (past the last column: behind everything)
  auto column = [&](int j) {
    const int col = (j * span + at) * 8;
    return LANES == 64 ? col : (col < g.d ? sub * g.d + col : 1 << 28);
  };
  auto read = [&](BackRow<S, V>& row, int64_t t) {
    const int sb = rows_at(t) * s_bytes, hb = rows_at(t) * h_bytes;
    const auto x = row_of(g.r, t * s_bytes, NEXT ? sb : 0), d = row_of(g.dr, t * s_bytes, g.dr != nullptr ? sb : 0);
    const auto dn = row_of(g.dn, t * h_bytes, NEXT ? hb : 0), more = row_of(g.dn_add, t * h_bytes, ADD ? hb : 0);
    const auto y = row_of(g.y, t * h_bytes, POST || CHANNEL || token ? hb : 0);
    if constexpr (BRANCH && !CHANNEL) {
      const auto gate = row_of(g.gate, t * 4, token ? rows_at(t) * 4 : 0);
      row.gate = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(gate, sub * 4, 0, 0));
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = column(j);
      if constexpr (NEXT) row.x[j].read(x, col), row.dn[j].read(dn, col);
      if constexpr (ADD) row.more[j].read(more, col);
      row.d[j].read(d, col);
      if constexpr (BRANCH) row.y[j].read(y, col);
    }
  };

  // a row is widened again for its second use: held in fp32 over the sums, it would spill
  constexpr bool kKeep = WIDE;
  int buf = 0;
  auto compute = [&](BackRow<S, V>& row, int64_t t) {
    // (the weights are read from LDS again for each use: kept over the rows, they would fill the registers)
    if constexpr (LANES < 64 || V > 1) asm volatile("" : : : "memory");
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * span + at) * 8;
      float wn[8], wp[8], gc[8];
      if constexpr (NEXT) weight(0, col, wn);
      if constexpr (POST) weight(kColPost, col, wp);
      if constexpr (CHANNEL) weight(kColGate, col, gc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float q = 0.0f;
        if constexpr (BRANCH) q = row.y[j][i];
        if constexpr (POST) {
          s[2] = fmaf(q, q, s[2]);
          q *= wp[i];
        }
        if constexpr (CHANNEL) q *= gc[i];
        if constexpr (BRANCH) s[3] = fmaf(q, row.d[j][i], s[3]);
        if constexpr (NEXT) {
          const float dn = ADD ? row.dn[j][i] + row.more[j][i] : row.dn[j][i], h = dn * wn[i], x = row.x[j][i];
          s[0] = fmaf(x, x, s[0]);
          s[1] = fmaf(h, x, s[1]);
          if constexpr (BRANCH) {
            s[4] = fmaf(q, h, s[4]);
            s[5] = fmaf(q, x, s[5]);
          }
        }
      }
      if constexpr (V > 1) {
#pragma unroll
        for (int i = 0; i < 6; ++i) asm volatile("" : "+v"(s[i]) : : "memory");
        __builtin_amdgcn_sched_barrier(0);  // one vector's weights at a time
      }
    }
    if (NEXT || POST || token) team_sum<LANES>(s, red, buf, waves, team * waves);
    const bool live = t + sub < g.T;
    // (a row that is not there has zeros for its sums: beside others in a wave no factor of it may be infinite)
    const bool there = LANES == 64 || live;
    const float k1 = NEXT && there ? rsqrtf(fmaf(s[0], inv_d, g.eps)) : 0.0f;
    const float k2 = k1 * s[1] * inv_d * k1 * k1;
    const float qg = s[3] + k1 * s[4] - k2 * s[5];  // sum of q g
    const float rsy = POST ? (there ? rsqrtf(fmaf(s[2], inv_d, g.eps)) : 0.0f) : 1.0f;
    float bt = g.b;
    if constexpr (BRANCH && !CHANNEL) bt = token ? g.b * row.gate : g.b;
    const float p1 = rsy * bt, p2 = rsy * qg * inv_d * rsy * rsy * bt;
    if (token && at == 0 && live) g.d_gate_token[t + sub] = g.b * rsy * qg;
    const auto dr_row = row_of(g.r_out, t * s_bytes, rows_at(t) * s_bytes);
    const auto dy_row = row_of(g.dy, t * h_bytes, BRANCH ? rows_at(t) * h_bytes : 0);
    if (t >= g.T) return;
    if constexpr (LANES < 64 || V > 1) asm volatile("" : : : "memory");
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * span + at) * 8;
      if constexpr (kKeep) {
        if constexpr (NEXT) row.x[j].keep(), row.dn[j].keep();
        if constexpr (ADD) row.more[j].keep();
        row.d[j].keep();
        if constexpr (BRANCH) row.y[j].keep();
      }
      float wn[8], wp[8], gc[8], dx[8], dy[8];
      if constexpr (NEXT) weight(0, col, wn);
      if constexpr (POST) weight(kColPost, col, wp);
      if constexpr (CHANNEL) weight(kColGate, col, gc);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float gr = row.d[j][i];
        if constexpr (NEXT) {
          const float dn = ADD ? row.dn[j][i] + row.more[j][i] : row.dn[j][i], x = row.x[j][i];
          gr = fmaf(k1, dn * wn[i], gr);
          gr = fmaf(-k2, x, gr);
          acc[0][j][i] = fmaf(dn, x * k1, acc[0][j][i]);
        }
        dx[i] = g.a * gr;
        if constexpr (BRANCH) {
          const float gated = CHANNEL ? gr * gc[i] : gr, y = row.y[j][i];
          if constexpr (POST) {
            acc[kColPost][j][i] = fmaf(p1 * gated, y, acc[kColPost][j][i]);
            dy[i] = fmaf(p1 * gated, wp[i], -p2 * y);
          } else {
            dy[i] = p1 * gated;
          }
          if constexpr (CHANNEL) {
            const float u = POST ? y * wp[i] : y;
            acc[kColGate][j][i] = fmaf(p1 * gr, u, acc[kColGate][j][i]);
          }
        }
      }
      write8(dr_row, column(j), dx, S{});
      if constexpr (BRANCH) write8(dy_row, column(j), dy, uint16_t{});
      if constexpr (LANES < 64 || V > 1) {
#pragma unroll
        for (int k = 0; k < kCols; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(acc[k][j][i]));  // added here, not put off behind the next row
      }
      if constexpr (V > 1) {
        asm volatile("" : : : "memory");
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // every workgroup's turn: rows t0 on, kRows of them a team; a team without a row goes along, for the barriers
  const int teams = WIDE ? 1 : __builtin_amdgcn_readfirstlane((int)blockDim.x / (64 * waves)), mine = team * kRows;
  const int64_t turn = (int64_t)gridDim.x * teams * kRows;
  int64_t t0 = (int64_t)blockIdx.x * teams * kRows;
  if constexpr (V > 1 || LANES < 64) {
    for (; t0 < g.T; t0 += turn) {
      BackRow<S, V> row;
      read(row, t0 + mine);
      compute(row, t0 + mine);
    }
  } else {
    BackRow<S, V> even, odd;
    read(even, t0 + mine);
    while (t0 < g.T) {
      read(odd, t0 + turn + mine);
      compute(even, t0 + mine);
      t0 += turn;
      if (t0 >= g.T) break;
      read(even, t0 + turn + mine);
      compute(odd, t0 + mine);
      t0 += turn;
    }
  }
  if constexpr (LANES < 64) {  // the rows of a wave
#pragma unroll
    for (int k = 0; k < kCols; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (LANES == 16) acc[k][0][i] = add_rows(acc[k][0][i]);
        acc[k][0][i] = add_halves(acc[k][0][i]);
      }
  }
  // the teams' sums, one after the other
  if constexpr (kCols > 0 && !WIDE) {
    __syncthreads();  // (the weights' last reads)
    for (int k = 1; k < teams; ++k) {
      if (team == k) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int j = 0; j < V; ++j) store8(w_lds + c * padded + (j * span + at) * 8, acc[c][j]);
      }
      __syncthreads();
      if (team == 0) {
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            float more[8];
            load8(w_lds + c * padded + (j * span + at) * 8, more);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[c][j][i] += more[i];
          }
      }
      __syncthreads();
    }
  }
  if (team == 0) {
#pragma unroll
    for (int k = 0; k < kCols; ++k) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * span + at) * 8;
        if (col < g.d) store8(g.partial + ((int64_t)blockIdx.x * kCols + k) * g.d + col, acc[k][j]);
      }
    }
  }
}

// out[c] = sum over groups of partial[group][k][c]: 64 columns a workgroup, the groups dealt to 16 waves,
// whose sums are joined in order.
constexpr int kSumWaves = 16;
struct ColumnSums {
  float* out[3];
};
__global__ __launch_bounds__(64 * kSumWaves) void column_sum_kernel(const float* __restrict__ partial, int groups,
                                                                    int cols, int d, ColumnSums o) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
  const int col = blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (col < d) {
    const float* p = partial + (int64_t)k * d + col;
    const int64_t pitch = (int64_t)cols * d;
#pragma unroll 8
    for (int i = wave; i < groups; i += kSumWaves) sum += p[i * pitch];
  }
  red[wave][lane] = sum;
  __syncthreads();
  float* out = o.out[k];
  if (wave == 0 && col < d && out != nullptr) {
    sum = red[0][lane];
#pragma unroll
    for (int w = 1; w < kSumWaves; ++w) sum += red[w][lane];
    out[col] = sum;
  }
}

// Lanes that hold a row of 8 columns each: a quarter or half of a wave for short rows, else whole waves (65536 x 64, bf16:
// with a wave a row 12.2, 25.3, 28.7 and 47.4 us for what takes 7.8, 9.7, 15.2 and 22.4 this way).
inline int row_lanes(int64_t d) { return d <= 128 ? 16 : (d <= 256 ? 32 : 64); }

// Waves of a team: V vectors of 8 columns a lane.
inline int vectors(int64_t d) { return d > 512 * kMaxWaves ? 2 : 1; }
inline int team_waves(int64_t d) {
  const int64_t per = 512 * vectors(d);
  return (int)((d + per - 1) / per);
}

template <class S, bool BRANCH, bool POST, bool NEXT>
hipError_t run_forward(const NormArgs& g, hipStream_t stream) {
  const int lanes = row_lanes(g.d), waves = lanes == 64 ? team_waves(g.d) : 4;
  const int64_t rows = lanes == 64 ? 1 : 64 / lanes * waves;  // of a workgroup's turn
  int64_t groups = (g.T + rows - 1) / rows;
  const int64_t fit = (int64_t)device_cu_count(current_device()) * (32 / waves);
  const dim3 grid((unsigned)(groups < fit ? groups : fit)), block(64 * waves);
  auto run = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, block, 0, stream, g);
    return hipGetLastError();
  };
  if (lanes == 16) return run(norm_kernel<S, BRANCH, POST, NEXT, 1, 16>);
  if (lanes == 32) return run(norm_kernel<S, BRANCH, POST, NEXT, 1, 32>);
  if (vectors(g.d) == 1) return run(norm_kernel<S, BRANCH, POST, NEXT, 1, 64>);
  return run(norm_kernel<S, BRANCH, POST, NEXT, 2, 64>);
}

template <class S>
hipError_t forward(const NormArgs& g, bool branch, bool post, bool next, hipStream_t stream) {
  if (!branch) return run_forward<S, false, false, true>(g, stream);
  if (post) return next ? run_forward<S, true, true, true>(g, stream) : run_forward<S, true, true, false>(g, stream);
  return next ? run_forward<S, true, false, true>(g, stream) : run_forward<S, true, false, false>(g, stream);
}

// Teams of a backward workgroup.
inline int back_teams(int64_t d) {
  const int fit = kBackWaves / team_waves(d);
  return fit > 1 ? fit : 1;
}

template <class S, bool BRANCH, bool POST, bool NEXT, bool CHANNEL, bool ADD>
hipError_t run_backward(const NormArgs& g, int groups, hipStream_t stream) {
  constexpr int kCols = (NEXT ? 1 : 0) + (POST ? 1 : 0) + (CHANNEL ? 1 : 0);
  const int teams = back_teams(g.d);
  const dim3 grid(groups), block(64 * g.team_waves * teams);
  const int lanes = row_lanes(g.d);
  // the weights; at the end a team's sums
  size_t lds = (size_t)kCols * g.team_waves * (lanes * 8) * vectors(g.d) * sizeof(float);
  if (lds > kBackLds) lds = 0;  // (V = 2 alone)
  auto run = [&](auto kernel) {
    if (lds > 64 * 1024) {
      const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                               kBackLds);
      if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, g);
    return hipGetLastError();
  };
  if (lanes == 16) return run(norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, ADD, false, 1, 16>);
  if (lanes == 32) return run(norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, ADD, false, 1, 32>);
  if (g.team_waves <= kBackWaves) return run(norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, ADD, false, 1, 64>);
  if (vectors(g.d) == 1) return run(norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, ADD, true, 1, 64>);
  return run(norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, ADD, true, 2, 64>);
}

template <class S, bool BRANCH, bool POST, bool NEXT, bool CHANNEL>
hipError_t backward_parts(const NormArgs& g, int groups, hipStream_t stream) {
  if constexpr (NEXT) {
    if (g.dn_add != nullptr) return run_backward<S, BRANCH, POST, NEXT, CHANNEL, true>(g, groups, stream);
  }
  return run_backward<S, BRANCH, POST, NEXT, CHANNEL, false>(g, groups, stream);
}

template <class S, bool POST, bool NEXT>
hipError_t backward_branch(const NormArgs& g, int groups, hipStream_t stream) {
  return g.gate_kind == MOE_GATE_CHANNEL ? backward_parts<S, true, POST, NEXT, true>(g, groups, stream)
                                         : backward_parts<S, true, POST, NEXT, false>(g, groups, stream);
}

template <class S>
hipError_t backward(const NormArgs& g, bool branch, bool post, bool next, int groups, hipStream_t stream) {
  if (!branch) return backward_parts<S, false, false, true, false>(g, groups, stream);
  if (post) return next ? backward_branch<S, true, true>(g, groups, stream) : backward_branch<S, true, false>(g, groups, stream);
  return next ? backward_branch<S, false, true>(g, groups, stream) : backward_branch<S, false, false>(g, groups, stream);
}

}  // namespace

// As many workgroups as are resident on 256 CUs: more partial rows would cost more than they overlap.
int64_t norm_partial_rows(int64_t T, int64_t d) {
  const int64_t rows = back_teams(d) * (64 / row_lanes(d));  // of a workgroup's turn
  const int64_t groups = (T + rows - 1) / rows, most = team_waves(d) > kBackWaves ? 256 : 512;
  return groups < most ? groups : most;
}

hipError_t launch_norm(const void* r, bool r_f32, const uint16_t* y, const void* w_post, const void* w_next,
                       const void* gate, int gate_kind, bool w_f32, bool post, bool next, float a, float b, float eps,
                       int64_t T, int64_t d, void* r_out, uint16_t* n_out, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  NormArgs g{};
  g.r = r, g.y = y, g.w_post = w_post, g.w_next = w_next, g.gate = gate, g.gate_kind = gate_kind, g.w_f32 = w_f32;
  g.a = a, g.b = b, g.eps = eps, g.T = T, g.d = (int)d, g.r_out = r_out, g.n_out = n_out;
  return r_f32 ? forward<float>(g, y != nullptr, post, next, stream)
               : forward<uint16_t>(g, y != nullptr, post, next, stream);
}

hipError_t launch_norm_backward(const void* dr, const uint16_t* dn, const uint16_t* dn_add, const uint16_t* y, const void* r,
                                bool r_f32, const void* w_post, const void* w_next, const void* gate, int gate_kind,
                                bool w_f32, bool branch, bool post, bool next, float a, float b, float eps, int64_t T, int64_t d,
                                void* dr_out, uint16_t* dy, float* d_gate, float* d_w_post, float* d_w_next,
                                float* partial, hipStream_t stream) {
  NormArgs g{};
  g.r = r, g.y = y, g.w_post = w_post, g.w_next = w_next, g.gate = gate, g.gate_kind = gate_kind, g.w_f32 = w_f32;
  g.a = a, g.b = b, g.eps = eps, g.T = T, g.d = (int)d, g.r_out = dr_out, g.dr = dr, g.dn = dn, g.dn_add = dn_add, g.dy = dy;
  g.d_gate_token = d_gate, g.partial = partial, g.team_waves = team_waves(d);
  const int groups = (int)norm_partial_rows(T, d);
  if (T > 0) {
    const hipError_t e = r_f32 ? backward<float>(g, branch, post, next, groups, stream)
                               : backward<uint16_t>(g, branch, post, next, groups, stream);
    if (e != hipSuccess) return e;
  }
  ColumnSums o{};
  int cols = 0;
  bool any = false;
  if (next) o.out[cols++] = d_w_next;
  if (post) o.out[cols++] = d_w_post;
  if (gate_kind == MOE_GATE_CHANNEL) o.out[cols++] = d_gate;
  for (int k = 0; k < cols; ++k) any = any || o.out[k] != nullptr;
  if (!any) return hipSuccess;
  hipLaunchKernelGGL(column_sum_kernel, dim3((unsigned)((d + 63) / 64), cols), dim3(64 * kSumWaves), 0, stream, partial,
                     groups, cols, (int)d, o);
  return hipGetLastError();
}

}  // namespace moe
