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
// consecutive columns (twice 8). The backward's teams walk the rows with the column sums in registers;
// each leaves one row of partial sums, which a second launch adds in order, so results repeat bit for bit.

#include "common.h"

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
  float* partial;        // [teams][sums][d]
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

// Sums over the whole team, the same in every lane. `buf` alternates between two LDS areas, so one
// barrier a round is enough: a wave reaches the round after next only behind the next one's barrier.
template <int N>
__device__ __forceinline__ void team_sum(float (&v)[N], float (*red)[kMaxWaves][N], int& buf, int waves) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[buf][wave][i] = v[i];
  }
  __syncthreads();
  const int from = lane & 15;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = sum16(from < waves ? red[buf][from][i] : 0.0f);
  buf ^= 1;
}

template <class S, bool BRANCH, bool POST, bool NEXT, int V>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_kernel(NormArgs g) {
  __shared__ float red[2][kMaxWaves][1];
  const int waves = blockDim.x >> 6;
  const S* r_in = static_cast<const S*>(g.r);
  S* r_out = static_cast<S*>(g.r_out);
  const float inv_d = 1.0f / (float)g.d;
  int buf = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const int64_t row = t * g.d;
    float x[V][8], u[V][8];
    float ss[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = u[j][i] = 0.0f;
      if (col < g.d) {
        load8(r_in + row + col, x[j]);
        if constexpr (BRANCH) load8(g.y + row + col, u[j]);
      }
    }
    if constexpr (BRANCH) {
      float scale = g.b;
      if (g.gate_kind == MOE_GATE_TOKEN) scale *= static_cast<const float*>(g.gate)[t];
      if constexpr (POST) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int i = 0; i < 8; ++i) ss[0] = fmaf(u[j][i], u[j][i], ss[0]);
        team_sum(ss, red, buf, waves);
        scale *= rsqrtf(fmaf(ss[0], inv_d, g.eps));
        ss[0] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
        if (col < g.d) {
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
      team_sum(ss, red, buf, waves);
      const float rs = rsqrtf(fmaf(ss[0], inv_d, g.eps));
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
        if (col < g.d) {
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

// CHANNEL: the gate is one per channel. The column sums stand in the order dw_next, dw_post, dgate, those
// that the form has.
template <class S, bool BRANCH, bool POST, bool NEXT, bool CHANNEL, int V>
__global__ __launch_bounds__(64 * kMaxWaves) void norm_backward_kernel(NormArgs g) {
  constexpr int kCols = (NEXT ? 1 : 0) + (POST ? 1 : 0) + (CHANNEL ? 1 : 0);
  constexpr int kColPost = NEXT ? 1 : 0, kColGate = kColPost + (POST ? 1 : 0);
  __shared__ float red[2][kMaxWaves][6];
  const int waves = blockDim.x >> 6;
  const S* x_in = static_cast<const S*>(g.r);
  const S* dr_in = static_cast<const S*>(g.dr);
  S* dr_out = static_cast<S*>(g.r_out);
  const float inv_d = 1.0f / (float)g.d;
  const bool token = BRANCH && g.gate_kind == MOE_GATE_TOKEN;
  float acc[kCols > 0 ? kCols : 1][V][8];
#pragma unroll
  for (int k = 0; k < kCols; ++k)
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[k][j][i] = 0.0f;
  int buf = 0;
  for (int64_t t = blockIdx.x; t < g.T; t += gridDim.x) {
    const int64_t row = t * g.d;
    float x[V][8], d[V][8], dn[V][8], y[V][8];
    float s[6] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = d[j][i] = dn[j][i] = y[j][i] = 0.0f;
      if (col < g.d) {
        if constexpr (NEXT) {
          load8(x_in + row + col, x[j]);
          load8(g.dn + row + col, dn[j]);
          if (g.dn_add != nullptr) {
            float more[8];
            load8(g.dn_add + row + col, more);
#pragma unroll
            for (int i = 0; i < 8; ++i) dn[j][i] += more[i];
          }
        }
        if (dr_in != nullptr) load8(dr_in + row + col, d[j]);
        if constexpr (POST || CHANNEL) load8(g.y + row + col, y[j]);
        else if (token) load8(g.y + row + col, y[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (col < g.d) {
        float wn[8], wp[8], gc[8];
        if constexpr (NEXT) load_weight(g.w_next, g.w_f32, col, wn);
        if constexpr (POST) load_weight(g.w_post, g.w_f32, col, wp);
        if constexpr (CHANNEL) load_weight(g.gate, g.w_f32, col, gc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float h = NEXT ? dn[j][i] * wn[i] : 0.0f;
          float q = y[j][i];
          if constexpr (POST) q *= wp[i];
          if constexpr (CHANNEL) q *= gc[i];
          if constexpr (NEXT) {
            s[0] = fmaf(x[j][i], x[j][i], s[0]);
            s[1] = fmaf(h, x[j][i], s[1]);
          }
          if constexpr (POST) s[2] = fmaf(y[j][i], y[j][i], s[2]);
          if constexpr (BRANCH) {
            s[3] = fmaf(q, d[j][i], s[3]);
            if constexpr (NEXT) {
              s[4] = fmaf(q, h, s[4]);
              s[5] = fmaf(q, x[j][i], s[5]);
            }
          }
        }
      }
    }
    if (NEXT || POST || token) team_sum(s, red, buf, waves);
    const float k1 = NEXT ? rsqrtf(fmaf(s[0], inv_d, g.eps)) : 0.0f;
    const float k2 = k1 * s[1] * inv_d * k1 * k1;
    const float qg = s[3] + k1 * s[4] - k2 * s[5];  // sum of q g
    const float rsy = POST ? rsqrtf(fmaf(s[2], inv_d, g.eps)) : 1.0f;
    const float bt = token ? g.b * static_cast<const float*>(g.gate)[t] : g.b;
    const float p1 = rsy * bt, p2 = rsy * qg * inv_d * rsy * rsy * bt;
    if (token && threadIdx.x == 0) g.d_gate_token[t] = g.b * rsy * qg;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (col < g.d) {
        float wn[8], wp[8], gc[8], dx[8], dy[8];
        if constexpr (NEXT) load_weight(g.w_next, g.w_f32, col, wn);
        if constexpr (POST) load_weight(g.w_post, g.w_f32, col, wp);
        if constexpr (CHANNEL) load_weight(g.gate, g.w_f32, col, gc);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float gr = d[j][i];
          if constexpr (NEXT) {
            gr = fmaf(k1, dn[j][i] * wn[i], gr);
            gr = fmaf(-k2, x[j][i], gr);
            acc[0][j][i] = fmaf(dn[j][i], x[j][i] * k1, acc[0][j][i]);
          }
          dx[i] = g.a * gr;
          if constexpr (BRANCH) {
            const float gated = CHANNEL ? gr * gc[i] : gr;
            if constexpr (POST) {
              acc[kColPost][j][i] = fmaf(p1 * gated, y[j][i], acc[kColPost][j][i]);
              dy[i] = fmaf(p1 * gated, wp[i], -p2 * y[j][i]);
            } else {
              dy[i] = p1 * gated;
            }
            if constexpr (CHANNEL) {
              const float u = POST ? y[j][i] * wp[i] : y[j][i];
              acc[kColGate][j][i] = fmaf(p1 * gr, u, acc[kColGate][j][i]);
            }
          }
        }
        store8(dr_out + row + col, dx);
        if constexpr (BRANCH) store8(g.dy + row + col, dy);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int col = (j * (int)blockDim.x + (int)threadIdx.x) * 8;
      if (col < g.d) store8(g.partial + ((int64_t)blockIdx.x * kCols + k) * g.d + col, acc[k][j]);
    }
  }
}

// out[c] = sum over teams of partial[team][k][c]: 64 columns a workgroup, the teams dealt to 16 waves,
// whose sums are joined in order.
constexpr int kSumWaves = 16;
struct ColumnSums {
  float* out[3];
};
__global__ __launch_bounds__(64 * kSumWaves) void column_sum_kernel(const float* __restrict__ partial, int teams,
                                                                    int cols, int d, ColumnSums o) {
  __shared__ float red[kSumWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, k = blockIdx.y;
  const int col = blockIdx.x * 64 + lane;
  float sum = 0.0f;
  if (col < d) {
    const float* p = partial + (int64_t)k * d + col;
    const int64_t pitch = (int64_t)cols * d;
#pragma unroll 8
    for (int i = wave; i < teams; i += kSumWaves) sum += p[i * pitch];
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

// Waves of a team: V vectors of 8 columns a lane.
inline int vectors(int64_t d) { return d > 512 * kMaxWaves ? 2 : 1; }
inline int team_waves(int64_t d) {
  const int64_t per = 512 * vectors(d);
  return (int)((d + per - 1) / per);
}

template <class S, bool BRANCH, bool POST, bool NEXT>
hipError_t run_forward(const NormArgs& g, hipStream_t stream) {
  const int waves = team_waves(g.d);
  int64_t teams = (int64_t)device_cu_count(current_device()) * (32 / waves);
  if (teams > g.T) teams = g.T;
  const dim3 grid((unsigned)teams), block(64 * waves);
  if (vectors(g.d) == 1) hipLaunchKernelGGL((norm_kernel<S, BRANCH, POST, NEXT, 1>), grid, block, 0, stream, g);
  else hipLaunchKernelGGL((norm_kernel<S, BRANCH, POST, NEXT, 2>), grid, block, 0, stream, g);
  return hipGetLastError();
}

template <class S>
hipError_t forward(const NormArgs& g, bool branch, bool post, bool next, hipStream_t stream) {
  if (!branch) return run_forward<S, false, false, true>(g, stream);
  if (post) return next ? run_forward<S, true, true, true>(g, stream) : run_forward<S, true, true, false>(g, stream);
  return next ? run_forward<S, true, false, true>(g, stream) : run_forward<S, true, false, false>(g, stream);
}

template <class S, bool BRANCH, bool POST, bool NEXT, bool CHANNEL>
hipError_t run_backward(const NormArgs& g, int teams, hipStream_t stream) {
  const dim3 grid(teams), block(64 * team_waves(g.d));
  if (vectors(g.d) == 1)
    hipLaunchKernelGGL((norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, 1>), grid, block, 0, stream, g);
  else
    hipLaunchKernelGGL((norm_backward_kernel<S, BRANCH, POST, NEXT, CHANNEL, 2>), grid, block, 0, stream, g);
  return hipGetLastError();
}

template <class S, bool POST, bool NEXT>
hipError_t backward_branch(const NormArgs& g, int teams, hipStream_t stream) {
  return g.gate_kind == MOE_GATE_CHANNEL ? run_backward<S, true, POST, NEXT, true>(g, teams, stream)
                                         : run_backward<S, true, POST, NEXT, false>(g, teams, stream);
}

template <class S>
hipError_t backward(const NormArgs& g, bool branch, bool post, bool next, int teams, hipStream_t stream) {
  if (!branch) return run_backward<S, false, false, true, false>(g, teams, stream);
  if (post) return next ? backward_branch<S, true, true>(g, teams, stream) : backward_branch<S, true, false>(g, teams, stream);
  return next ? backward_branch<S, false, true>(g, teams, stream) : backward_branch<S, false, false>(g, teams, stream);
}

}  // namespace

int64_t norm_partial_rows(int64_t T, int64_t d) {
  const int64_t most = 32 / team_waves(d) < 3 ? 512 : 768;
  return T < most ? T : most;
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
  g.d_gate_token = d_gate, g.partial = partial;
  const int teams = (int)norm_partial_rows(T, d);
  if (T > 0) {
    const hipError_t e = r_f32 ? backward<float>(g, branch, post, next, teams, stream)
                               : backward<uint16_t>(g, branch, post, next, teams, stream);
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
                     teams, cols, (int)d, o);
  return hipGetLastError();
}

}  // namespace moe
