// Router of the MoE layer: from logits x [T, E] the k routed experts of every token, their weights,
// and, for training, the balance loss, the z-loss and the gradient of the logits.
//
//   m = max_i x_i,  s = sum_i exp(x_i - m),  lse = m + log s,  p_i = exp(x_i - m) / s
//   ids = the k largest logits, the lowest index first among equals; -inf is never chosen
//   w_j = p_{id_j}, or p_{id_j} / sum_l p_{id_l} (renormalised)
//   losses = ( E sum_e f_e P_e , 1/n sum_t lse_t^2 ),  f_e = counts_e / sum counts,  P_e = 1/n sum_t p_te
//
// over the n tokens whose row is not all -inf. With c_e = dL0 E f_e / n the gradient of a row is
//
//   dx_i = p_i (c_i - sum_l c_l p_l + 2 dL1 lse / n) + routing part,
//   routing part = w_j (g_j - sum_l g_l w_l) at i = id_j (renormalised), else p_i (g_i - sum_l g_l p_{id_l})
//
// with g the gradient of the weights (g_i zero off the chosen experts).
//
// G lanes hold one token (V consecutive experts each), so a wave works on 64 / G tokens and a
// reduction over a token is log2 G lane exchanges. The row stays in registers from its one read to
// its last use. Everything is fp32; rows are summed in a fixed order, and column sums over tokens go
// lane -> workgroup -> a second launch over the workgroups' partials, also in a fixed order.
//
// Small calls are bound by latency (one read, log2 G exchanges a reduction, k rounds), large ones by issuing
// instructions: a logit costs about 20 for its key and exponential and 8 per round of selection. Measured: 4
// tokens of 128 experts 4.1 us, 8192 x 64 5.1; 65537 x 100 fp32, top-6, selection 16.9 us, with the losses
// 23.2 + 5.4, gradient 15.5 (3.4 TB/s; a profiler's times, about a microsecond a launch above those of calls back
// to back). The second launch stands because a call's workspace may hold anything: a last workgroup that adds the
// partial sums would count arrivals in it, which asks for a workspace zeroed once (it could set the count back itself).

#include <type_traits>

#include "common.h"

namespace moe {
namespace {

constexpr int kPlainThreads = 256;
// With the losses a workgroup leaves one partial sum per column, and the second launch adds them in
// one workgroup: at most one large workgroup a CU, of 8 waves while those hold all tokens at once, of
// 16 beyond. Both launches of 65537 tokens of 100 experts 28 us (two workgroups of 8 waves a CU: 30,
// one: 34), of 8192 tokens of 256 experts 18.7 us (24 and 20), of 4096 tokens of 128 experts (8 waves,
// 128 workgroups) 11.4 us (16 waves: 12.7).
constexpr int64_t kLossBlocks = 256;
constexpr int kLossThreads = 512, kLossThreadsMany = 1024;

__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Value of the lane whose index differs from this one's in the bits of a group step: lanes 1, 2
// (quad permutes), 4 (mirror of 8, after the quads agree), 8 (mirror of 16), 16 and 32 apart.
template <int STEP>
__device__ __forceinline__ float partner(float v) {
  if constexpr (STEP == 1) return dpp<0xB1>(v);
  else if constexpr (STEP == 2) return dpp<0x4E>(v);
  else if constexpr (STEP == 4) return dpp<0x141>(v);
  else if constexpr (STEP == 8) return dpp<0x140>(v);
  else return __shfl_xor(v, STEP, 64);
}

template <int STEP>
__device__ __forceinline__ int partner(int v) { return __float_as_int(partner<STEP>(__int_as_float(v))); }

// Maximum and sum over the G lanes of a token, the same value in all of them. (The mirrors pair
// lanes of halves that already agree, and a + b = b + a, so every lane forms the same sum.)
template <int G, typename T>
__device__ __forceinline__ T group_max(T v) {
  v = max(v, partner<1>(v));
  v = max(v, partner<2>(v));
  v = max(v, partner<4>(v));
  if constexpr (G > 8) v = max(v, partner<8>(v));
  if constexpr (G > 16) v = max(v, partner<16>(v));
  if constexpr (G > 32) v = max(v, partner<32>(v));
  return v;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
  v += partner<1>(v);
  v += partner<2>(v);
  v += partner<4>(v);
  if constexpr (G > 8) v += partner<8>(v);
  if constexpr (G > 16) v += partner<16>(v);
  if constexpr (G > 32) v += partner<32>(v);
  return v;
}

// Logits as integers in the same order (two's complement of the magnitude for negative ones), so that
// maxima and comparisons need no care for NaNs: those, and the places past E, become -inf, which is
// never chosen. -0 becomes 0, its equal.
constexpr int kNegInfKey = (int)0x807FFFFFu;

__device__ __forceinline__ int order_key(float v) {
  const int i = __float_as_int(v + 0.f);
  return v == v ? i ^ ((i >> 31) & 0x7FFFFFFF) : kNegInfKey;
}

// e^x for x <= 0: with t = x log2 e = n + f, n whole, e^x = 2^n 2^f. The rounding of t and of log2 e
// is put back into f (Cody and Waite's reduction: log2 e as the nearest float and the float nearest its
// remainder), and the scaling by 2^n keeps results below 2^-126, which the hardware's exponential alone would flush. Off by under two units in the last place like the library's, in 11
// instructions instead of over 20. Below -200 the result is 0 in any case; a NaN stays one.
__device__ __forceinline__ float exp_nonpositive(float x) {
  x = x < -200.f ? -200.f : x;
  constexpr float kLog2e = 1.44269502162933349609375f, kRest = 1.925963033500011079e-8f;
  const float t = x * kLog2e;
  const float n = rintf(t);
  const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -t));
  return ldexpf(__builtin_amdgcn_exp2f((t - n) + rest), (int)n);
}

// This lane's V logits of row t, -inf past E. `wide`: rows start on 16 bytes and E is a whole
// number of 16-byte chunks.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* x, int64_t t, int E, int e0, bool wide, float (&v)[V]) {
  const T* row = x + t * E;
  constexpr int kChunk = 16 / sizeof(T);
  if (wide) {
#pragma unroll
    for (int c = 0; c < V / kChunk; ++c) {
      if (e0 + c * kChunk < E) {
        const u32x4 r = *reinterpret_cast<const u32x4*>(row + e0 + c * kChunk);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (sizeof(T) == 2) {
            v[c * 8 + 2 * q] = bf16_bits_to_f32(r[q] & 0xFFFFu);
            v[c * 8 + 2 * q + 1] = bf16_bits_to_f32(r[q] >> 16);
          } else {
            v[c * 4 + q] = __uint_as_float(r[q]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c * kChunk + i] = neg_inf();
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      v[i] = neg_inf();
      if (e0 + i < E) {
        if constexpr (sizeof(T) == 2) v[i] = bf16_bits_to_f32(row[e0 + i]);
        else v[i] = row[e0 + i];
      }
    }
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* x, int64_t t, int E, int e0, bool wide, const float (&v)[V]) {
  T* row = x + t * E;
  constexpr int kChunk = 16 / sizeof(T);
  if (wide) {
#pragma unroll
    for (int c = 0; c < V / kChunk; ++c) {
      if (e0 + c * kChunk < E) {
        u32x4 r;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (sizeof(T) == 2) r[q] = pack_bf16x2(v[c * 8 + 2 * q], v[c * 8 + 2 * q + 1]);
          else r[q] = __builtin_bit_cast(uint32_t, v[c * 4 + q]);
        }
        *reinterpret_cast<u32x4*>(row + e0 + c * kChunk) = r;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (e0 + i < E) {
        if constexpr (sizeof(T) == 2) row[e0 + i] = f32_to_bf16_bits(v[i]);
        else row[e0 + i] = v[i];
      }
  }
}

// exp(x_i - m0) of this lane's logits and their sum over the row.
template <int G, int V>
__device__ __forceinline__ float exponentials_from(const float (&v)[V], float m0, float (&e)[V]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    e[i] = exp_nonpositive(v[i] - m0);  // a NaN logit reaches the sum here
    s += e[i];
  }
  return group_sum<G>(s);
}

// exp(x_i - m) of this lane's logits and their sum over the row, and the logits' keys. A row of -inf
// alone has m = -inf; it is shifted by 0 instead, so that its exponentials and sum are 0 and its lse -inf.
template <int G, int V>
__device__ __forceinline__ float row_exponentials(const float (&v)[V], float& m0, float (&e)[V], int (&key)[V]) {
  int top = kNegInfKey;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    key[i] = order_key(v[i]);
    top = max(top, key[i]);
  }
  top = group_max<G>(top);
  m0 = top == kNegInfKey ? 0.f : __int_as_float(top ^ ((top >> 31) & 0x7FFFFFFF));
  return exponentials_from<G, V>(v, m0, e);
}

// The same without the keys.
template <int G, int V>
__device__ __forceinline__ float row_exponentials(const float (&v)[V], float& m0, float (&e)[V]) {
  float top = neg_inf();
#pragma unroll
  for (int i = 0; i < V; ++i) top = fmaxf(top, v[i]);  // a NaN loses
  top = group_max<G>(top);
  m0 = top == neg_inf() ? 0.f : top;
  return exponentials_from<G, V>(v, m0, e);
}

struct RouterArgs {
  const void* logits;
  int64_t T;
  int E, k;
  bool renormalize, wide;
  int32_t* ids;
  float* w;
  float* lse;
  uint32_t* partial;  // losses only: per workgroup E column sums, E counts, the sum of lse^2, the tokens
};

// Words of a workgroup's partial sums, padded to whole 16 bytes.
__host__ __device__ constexpr int64_t partial_words(int E) { return (2 * (int64_t)E + 2 + 3) / 4 * 4; }

template <typename T, int G, int V, bool LOSSES, int kThreads>
__global__ __launch_bounds__(kThreads) void router_topk_kernel(RouterArgs a) {
  constexpr int kGroups = kThreads / G;  // tokens a workgroup holds at once
  constexpr int kSlots = MOE_ROUTER_MAX_TOPK;
  constexpr int kSelWords = 2 * kGroups * kSlots, kSumWords = LOSSES ? kGroups * G * V : 1;
  __shared__ uint32_t shared_words[kSelWords > kSumWords ? kSelWords : kSumWords];
  float (*sel_part)[kSlots] = reinterpret_cast<float (*)[kSlots]>(shared_words);
  int (*sel_id)[kSlots] = reinterpret_cast<int (*)[kSlots]>(shared_words + kGroups * kSlots);
  float* colsum = reinterpret_cast<float*>(shared_words);  // behind the last token
  __shared__ int hist[LOSSES ? G * V : 1];
  __shared__ float zsum_s[LOSSES ? kGroups : 1];
  __shared__ int tokens_s[LOSSES ? kGroups : 1];
  const int tid = threadIdx.x, group = tid / G, g = tid % G, lane = tid & 63;
  const uint64_t below = ((1ull << lane) - 1) & ~((1ull << (lane - g)) - 1);  // the group's lanes below this one
  const int e0 = g * V;
  float col[V];
  float zsum = 0.f;
  int tokens = 0;
  if constexpr (LOSSES) {
    for (int e = tid; e < G * V; e += kThreads) hist[e] = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) col[i] = 0.f;
    __syncthreads();
  }
  const int64_t stride = (int64_t)gridDim.x * kGroups;
  float next[V];  // the next token's row, asked for while this one is worked on
  if ((int64_t)blockIdx.x * kGroups + group < a.T)
    load_row<T, V>(static_cast<const T*>(a.logits), (int64_t)blockIdx.x * kGroups + group, a.E, e0, a.wide, next);
  for (int64_t t = (int64_t)blockIdx.x * kGroups + group; t < a.T; t += stride) {
    float v[V], ex[V];
    int key[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    if (t + stride < a.T) load_row<T, V>(static_cast<const T*>(a.logits), t + stride, a.E, e0, a.wide, next);
    float m0;
    const float s = row_exponentials<G, V>(v, m0, ex, key);
    const float lse = m0 + logf(s);
    if (g == 0) a.lse[t] = lse;
    if constexpr (LOSSES) {
      if (s != 0.f) {  // NaN rows count and carry their NaN
        const float inv = 1.f / s;
#pragma unroll
        for (int i = 0; i < V; ++i) col[i] += ex[i] * inv;
        if (g == 0) {
          zsum += lse * lse;
          ++tokens;
        }
      }
    }
    // k rounds of: the row's largest remaining logit, the lowest lane that holds it, its lowest index there
    for (int j = 0; j < a.k; ++j) {
      int best = kNegInfKey;
#pragma unroll
      for (int i = 0; i < V; ++i) best = max(best, key[i]);
      const int top = group_max<G>(best);
      const uint64_t have = __ballot(best == top);
      if (best == top && (have & below) == 0) {
        int at = -1;
        float part = 0.f;
        bool found = top == kNegInfKey;  // none is left
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const bool hit = !found && key[i] == top;
          at = hit ? e0 + i : at;
          part = hit ? ex[i] : part;
          key[i] = hit ? kNegInfKey : key[i];
          found |= hit;
        }
        sel_id[group][j] = at;
        sel_part[group][j] = part;
        if constexpr (LOSSES) {
          if (at >= 0) atomicAdd(&hist[at], 1);  // LDS integer atomics: order-free
        }
      }
    }
    // the group's lanes are of one wave: its LDS writes above are complete once waited for
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_wave_barrier();
    float denom = s;
    if (a.renormalize) {
      float chosen = 0.f;
      for (int j = g; j < a.k; j += G) chosen += sel_part[group][j];
      chosen = group_sum<G>(chosen);
      denom = s == s ? chosen : s;
    }
    for (int j = g; j < a.k; j += G) {
      const int id = sel_id[group][j];
      a.ids[t * a.k + j] = id;
      a.w[t * a.k + j] = id < 0 ? 0.f : sel_part[group][j] / denom;
    }
    __builtin_amdgcn_s_waitcnt(0xC07F);
    __builtin_amdgcn_wave_barrier();
  }
  if constexpr (LOSSES) {
    __syncthreads();  // every group is done with its selection
#pragma unroll
    for (int i = 0; i < V; ++i) colsum[group * (G * V) + e0 + i] = col[i];
    if (g == 0) {
      zsum_s[group] = zsum;
      tokens_s[group] = tokens;
    }
    __syncthreads();
    uint32_t* out = a.partial + blockIdx.x * partial_words(a.E);
    for (int e = tid; e < a.E; e += kThreads) {
      float sum = 0.f;
#pragma unroll 16
      for (int q = 0; q < kGroups; ++q) sum += colsum[q * (G * V) + e];
      out[e] = __builtin_bit_cast(uint32_t, sum);
      out[a.E + e] = (uint32_t)hist[e];
    }
    if (tid == 0) {
      float z = 0.f;
      int n = 0;
#pragma unroll 16
      for (int q = 0; q < kGroups; ++q) {
        z += zsum_s[q];
        n += tokens_s[q];
      }
      out[2 * a.E] = __builtin_bit_cast(uint32_t, z);
      out[2 * a.E + 1] = (uint32_t)n;
      for (int w = 2 * a.E + 2; w < (int)partial_words(a.E); ++w) out[w] = 0u;
    }
  }
}

// The workgroups' partial sums to counts, tokens, P and the two losses: one workgroup. A thread adds
// four neighbouring words (16-byte loads, sixteen in flight) of every R-th partial in order, then a
// word's R slice sums are added in order, so the result does not depend on scheduling.
constexpr int kFinishThreads = 1024;

__global__ __launch_bounds__(kFinishThreads) void router_losses_kernel(const uint32_t* __restrict__ partial, int blocks,
                                                                       int E, int32_t* __restrict__ counts,
                                                                       int32_t* __restrict__ tokens,
                                                                       float* __restrict__ prob_mean,
                                                                       float* __restrict__ losses) {
  __shared__ u32x4 slice_sum[kFinishThreads];
  __shared__ float wave_f[kFinishThreads / 64];
  __shared__ int wave_i[kFinishThreads / 64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int quads = (int)(partial_words(E) / 4);
  constexpr int kBatch = 16;
  const int R = min(kFinishThreads / quads, (blocks + kBatch - 1) / kBatch);  // slices (quads <= 513)
  const int quad = tid % quads, slice = tid / quads;
  const u32x4* src = reinterpret_cast<const u32x4*>(partial);
  auto is_float = [&](int w) { return w < E || w == 2 * E; };  // P sums and the sum of lse^2; else counts and tokens
  float f[4] = {0.f, 0.f, 0.f, 0.f};
  uint32_t c[4] = {0u, 0u, 0u, 0u};
  if (slice < R) {
    for (int b0 = slice; b0 < blocks; b0 += R * kBatch) {
      u32x4 v[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        v[u] = b0 + u * R < blocks ? src[(int64_t)(b0 + u * R) * quads + quad] : u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          f[w] += __uint_as_float(v[u][w]);  // one of the two is not used
          c[w] += v[u][w];
        }
    }
    u32x4 out;
#pragma unroll
    for (int w = 0; w < 4; ++w) out[w] = is_float(4 * quad + w) ? __float_as_uint(f[w]) : c[w];
    slice_sum[slice * quads + quad] = out;
  }
  __syncthreads();
  // the slices' sums in order: of this thread's expert, and of lse^2 and the tokens (neighbouring words)
  const uint32_t* words = reinterpret_cast<const uint32_t*>(slice_sum);
  const int expert = tid < E ? tid : 0;
  float p_sum = 0.f, z_sum = 0.f;
  int count = 0, n = 0;
#pragma unroll 8
  for (int q = 0; q < R; ++q) {
    const uint32_t* at = words + q * quads * 4;
    const uint2 zn = *reinterpret_cast<const uint2*>(at + 2 * E);
    p_sum += __uint_as_float(at[expert]);
    count += (int)at[E + expert];
    z_sum += __uint_as_float(zn.x);
    n += (int)zn.y;
  }
  const float nf = (float)(n > 0 ? n : 1);
  const float mean = tid < E ? p_sum / nf : 0.f;
  if (tid < E) {
    counts[tid] = count;
    prob_mean[tid] = mean;
  } else {
    count = 0;
  }
  // sum of counts and of counts_e P_e over the experts
  float dot = (float)count * mean;
  int total = count;
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    dot += __shfl_xor(dot, off, 64);
    total += __shfl_xor(total, off, 64);
  }
  if (lane == 0) {
    wave_f[wave] = dot;
    wave_i[wave] = total;
  }
  __syncthreads();
  if (tid == 0) {
    dot = 0.f;
    total = 0;
    for (int q = 0; q < kFinishThreads / 64; ++q) {
      dot += wave_f[q];
      total += wave_i[q];
    }
    tokens[0] = n;
    losses[0] = (float)E * dot / (float)(total > 0 ? total : 1);
    losses[1] = z_sum / nf;
  }
}

struct RouterBackwardArgs {
  const void* logits;
  int64_t T;
  int E, k;
  bool renormalize, wide;
  const int32_t* ids;
  const float* w;
  const int32_t* counts;  // these two are read for the gradient of the losses alone
  const int32_t* tokens;
  const float* d_w;       // null: no gradient of the weights
  const float* d_losses;  // null: no gradient of the losses
  void* d_logits;
};

template <typename T, int G, int V>
__global__ __launch_bounds__(kPlainThreads) void router_backward_kernel(RouterBackwardArgs a) {
  constexpr int kGroups = kPlainThreads / G;
  // the routing part of a token's gradient, expert by expert: every chosen slot adds to its expert's
  // place, and the lane that holds the expert reads it
  __shared__ __align__(16) float routing[kGroups][G * V];
  const int tid = threadIdx.x, group = tid / G, g = tid % G;
  const int e0 = g * V;
  const int64_t stride = (int64_t)gridDim.x * kGroups;
  int64_t t = (int64_t)blockIdx.x * kGroups + group;
  // a token's row and this lane's first slot of it, asked for one token ahead
  float next[V];
  int next_id = -1;
  float next_g = 0.f, next_w = 0.f;
  auto fetch = [&](int64_t at) {
    load_row<T, V>(static_cast<const T*>(a.logits), at, a.E, e0, a.wide, next);
    if (a.d_w != nullptr && g < a.k) {
      next_id = a.ids[at * a.k + g];
      next_g = a.d_w[at * a.k + g];
      next_w = a.w[at * a.k + g];
    }
  };
  if (t < a.T) fetch(t);
  // c_e = dL0 E f_e / n of this lane's experts, and 2 dL1 / n
  float c[V], dz = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 0.f;
  if (a.d_losses != nullptr) {
    const int n = a.tokens[0];
    const float d0 = a.d_losses[0], d1 = a.d_losses[1];
    // every lane of a group holds a part of the counts: their sum is the group's (64 bits: over a batch of several
    // ranks the slots of all experts together pass 2^31 before the tokens do)
    int counts[V];
    long long total = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) counts[i] = a.counts[e0 + i < a.E ? e0 + i : 0];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      counts[i] = e0 + i < a.E ? counts[i] : 0;
      total += counts[i];
    }
#pragma unroll
    for (int off = 1; off < G; off <<= 1) total += __shfl_xor(total, off, 64);
    const float nf = (float)(n > 0 ? n : 1);
    const float scale = d0 * (float)a.E / ((float)(total > 0 ? total : 1) * nf);
    dz = 2.f * d1 / nf;
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = (float)counts[i] * scale;
  }
  for (; t < a.T; t += stride) {
    float v[V], p[V], d[V];
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = next[i];
    const int id = next_id;
    const float slot_g = next_g, slot_w = next_w;
    if (t + stride < a.T) fetch(t + stride);
    float m0;
    const float s = row_exponentials<G, V>(v, m0, p);
    if (s == 0.f) {  // nothing to choose from: no probability, no gradient
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.f;
      store_row<T, V>(static_cast<T*>(a.d_logits), t, a.E, e0, a.wide, d);
      continue;
    }
    const float inv = 1.f / s;
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      p[i] *= inv;
      dot += c[i] * p[i];
    }
    dot = group_sum<G>(dot);
    float shift = dz * (m0 + logf(s)) - dot;
    float part[V];
#pragma unroll
    for (int i = 0; i < V; ++i) part[i] = 0.f;
    if (a.d_w != nullptr) {
      float* row = routing[group];
#pragma unroll
      for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(row + e0 + i) = float4{0.f, 0.f, 0.f, 0.f};
      float gw = 0.f;  // sum over the kept slots of g_j w_j
      if (g < a.k && (unsigned)id < (unsigned)a.E) gw = slot_g * slot_w;
      for (int j = g + G; j < a.k; j += G) {
        const int at = a.ids[t * a.k + j];
        if ((unsigned)at < (unsigned)a.E) gw += a.d_w[t * a.k + j] * a.w[t * a.k + j];
      }
      gw = group_sum<G>(gw);
      // distinct ids: one addend each
      if (g < a.k && (unsigned)id < (unsigned)a.E) atomicAdd(row + id, slot_w * (a.renormalize ? slot_g - gw : slot_g));
      for (int j = g + G; j < a.k; j += G) {
        const int at = a.ids[t * a.k + j];
        if ((unsigned)at < (unsigned)a.E)
          atomicAdd(row + at, a.w[t * a.k + j] * (a.renormalize ? a.d_w[t * a.k + j] - gw : a.d_w[t * a.k + j]));
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the group is of one wave
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(row + e0 + i);
        part[i] = v.x; part[i + 1] = v.y; part[i + 2] = v.z; part[i + 3] = v.w;
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);
      __builtin_amdgcn_wave_barrier();
      if (!a.renormalize) shift -= gw;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) d[i] = p[i] * (c[i] + shift) + part[i];
    store_row<T, V>(static_cast<T*>(a.d_logits), t, a.E, e0, a.wide, d);
  }
}

// Workgroups of a launch over T tokens, kGroups at a time.
int64_t router_blocks(int64_t T, int groups, int64_t cap) {
  const int64_t blocks = (T + groups - 1) / groups;
  return blocks < 1 ? 1 : (blocks > cap ? cap : blocks);
}

// Lanes per token: 8 experts a lane up to 512 experts, 16 beyond. (16 a lane also for 65537 tokens of 100
// experts: selection with its sums 21.0 instead of 22.4 us, gradient 19.2 instead of the 17.3 it took then.)
int lanes_of(int E) { return E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 32 : 64; }

int loss_threads(int64_t T, int E) { return T * lanes_of(E) <= kLossBlocks * kLossThreads ? kLossThreads : kLossThreadsMany; }

int64_t loss_blocks(int64_t T, int E) { return router_blocks(T, loss_threads(T, E) / lanes_of(E), kLossBlocks); }

template <typename F>
hipError_t by_width(int E, F&& f) {
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 8>{});
  if (E <= 256) return f(std::integral_constant<int, 32>{}, std::integral_constant<int, 8>{});
  if (E <= 512) return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 64>{}, std::integral_constant<int, 16>{});
}

bool wide_rows(const void* p, int E, bool f32) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && E % (f32 ? 4 : 8) == 0;
}

}  // namespace

int64_t router_partial_words(int64_t T, int32_t E) {
  return loss_blocks(T, E) * partial_words(E);
}

hipError_t launch_router_topk(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renormalize,
                              int32_t* ids, float* w, float* lse, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const RouterArgs a{logits, T, E, k, renormalize, wide_rows(logits, E, f32), ids, w, lse, nullptr};
  const int64_t cap = (int64_t)device_cu_count(current_device()) * 16;
  return by_width(E, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    const dim3 grid((unsigned)router_blocks(T, kPlainThreads / G, cap));
    if (f32) hipLaunchKernelGGL((router_topk_kernel<float, G, V, false, kPlainThreads>), grid, dim3(kPlainThreads), 0, stream, a);
    else hipLaunchKernelGGL((router_topk_kernel<uint16_t, G, V, false, kPlainThreads>), grid, dim3(kPlainThreads), 0, stream, a);
    return hipGetLastError();
  });
}

hipError_t launch_router_topk_losses(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renormalize,
                                     int32_t* ids, float* w, float* lse, int32_t* counts, int32_t* tokens,
                                     float* prob_mean, float* losses, uint32_t* partial, hipStream_t stream) {
  const RouterArgs a{logits, T, E, k, renormalize, wide_rows(logits, E, f32), ids, w, lse, partial};
  const int64_t blocks = loss_blocks(T, E);
  const bool many = loss_threads(T, E) == kLossThreadsMany;
  const hipError_t st = by_width(E, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    auto launch = [&](auto kernel, int threads) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)blocks), dim3(threads), 0, stream, a);
      return hipGetLastError();
    };
    if (f32) return many ? launch(router_topk_kernel<float, G, V, true, kLossThreadsMany>, kLossThreadsMany)
                         : launch(router_topk_kernel<float, G, V, true, kLossThreads>, kLossThreads);
    return many ? launch(router_topk_kernel<uint16_t, G, V, true, kLossThreadsMany>, kLossThreadsMany)
                : launch(router_topk_kernel<uint16_t, G, V, true, kLossThreads>, kLossThreads);
  });
  if (st != hipSuccess) return st;
  hipLaunchKernelGGL(router_losses_kernel, dim3(1), dim3(kFinishThreads), 0, stream, partial, (int)blocks, E, counts,
                     tokens, prob_mean, losses);
  return hipGetLastError();
}

hipError_t launch_router_backward(const void* logits, bool f32, int64_t T, int32_t E, int32_t k, bool renormalize,
                                  const int32_t* ids, const float* w, const int32_t* counts, const int32_t* tokens,
                                  const float* d_w, const float* d_losses, void* d_logits, hipStream_t stream) {
  if (T == 0) return hipSuccess;
  const bool wide = wide_rows(logits, E, f32) && wide_rows(d_logits, E, f32);
  const RouterBackwardArgs a{logits, T, E, k, renormalize, wide, ids, w, counts, tokens, d_w, d_losses, d_logits};
  // Three workgroups a CU: each waits once for the counts, then walks the tokens with the next row on its way. 65537
  // tokens, us with 2 / 3 / 4 / 6 / 8 a CU: 100 experts fp32 15.5 / 14.7 / 15.1 / 15.3 / 16.9, bf16 25.9 / 23.8 / 22.7 /
  // 22.6 / 27.0 (rows of 100 bf16 are read two bytes at a time); 32 bf16 8.5 / 7.6 / 7.6 / 7.4 / 8.0; 64 fp32 11.6 / 10.9 /
  // 11.5 / 11.3 / 11.7; 128 bf16 17.2 / 16.0 / 16.1 / 16.2 / 17.7; 256 fp32 27.9 / 26.6 / 26.9 / 26.7 / 27.8; 512 bf16 56.4 /
  // 45.2 / 41.6 / 38.4 / 40.6; 1000 fp32 136 / 143 / 144 / 146 / 146; 8192 tokens of 512 bf16 10.8 / 9.9 / 10.6 / 10.6 / 13.0.
  const int64_t cap = (int64_t)device_cu_count(current_device()) * 3;
  return by_width(E, [&](auto g, auto v) {
    constexpr int G = decltype(g)::value, V = decltype(v)::value;
    const dim3 grid((unsigned)router_blocks(T, kPlainThreads / G, cap));
    if (f32) hipLaunchKernelGGL((router_backward_kernel<float, G, V>), grid, dim3(kPlainThreads), 0, stream, a);
    else hipLaunchKernelGGL((router_backward_kernel<uint16_t, G, V>), grid, dim3(kPlainThreads), 0, stream, a);
    return hipGetLastError();
  });
}

}  // namespace moe
