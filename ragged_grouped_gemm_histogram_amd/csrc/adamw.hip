// One AdamW step over a list of tensors, one launch per kListed tensors. For a value p with gradient g:
//
//   m = b1 m + (1 - b1) g      v = b2 v + (1 - b2) g^2
//   p = (1 - lr wd) p - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// all in fp32 (gradients are read as they are, parameters from their fp32 copy where there is one). Bound
// by HBM: 28 bytes a value with bf16 parameters, fp32 copies and moments, 10 with 8-bit moments alone. Measured, bf16
// parameters and gradients: 398 M values with fp32 copies and moments 2174 us (5.1 TB/s; a copy of 2 GiB runs at 4.9),
// 302 M with 8-bit moments and random rounding 565 to 585 us (5.2 to 5.4 TB/s), the moments' values as bf16 370 (5.0). With
// 32-bit moments and no copy 302 M bf16 parameters take 1291 us (5.1 TB/s, rounded at random 1467, 4.5), fp32 ones 1562 (5.4).
// Steps that brought it there: a pass's loads before the step of the one before, 2268 to 2215 and 743 to 616 us; whole
// lines read and written past the caches, 2215 to 2175 and 616 to 575.
//
// Moments in 8 bits: 32 consecutive values share a power of two 2^(byte - 127). The first moment is
// float8 e4m3, the block's largest magnitude in [128, 256) so that nothing saturates, to nearest even. The
// second needs range and no sign: code c stands for (1 + (c % 8) / 8) 2^(c / 8), 0 for c = 0, the largest
// with c / 8 = 30; anything above zero keeps at least code 1, so that a small second moment never
// vanishes under its first. Both scale by powers of two alone and the moments are taken in separate,
// unfused operations, so that the codes are determined to the bit. With (1 - b2) far below a code's step
// rounding to nearest would hold v where it is: a seed makes its rounding random, with a mean of v.
// The step itself uses m and v before they are rounded. A block with an infinity or a NaN gets byte 255
// and reads as NaN.

#include <cmath>

#include "common.h"

// Sums and products of the moments are rounded one by one.
#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kListed = 80;  // tensors per launch: their table travels in the kernel's arguments (4 KB)
constexpr int kPer = 8;      // consecutive values of a thread
constexpr int kPass = kThreads * kPer;  // values of a workgroup's step; a chunk is one or two, within one tensor

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct Listed {
  void* param;
  const void* grad;
  int64_t n;
  int64_t at;       // first value's place in the moments
  int32_t flags;
  int32_t pad;
};
constexpr double kLeastEps = 1e-12;  // see adamw_kernel
constexpr int kParamF32 = 1, kGradF32 = 2, kParamAligned = 4, kGradAligned = 8;

struct AdamArgs {
  void* m;
  uint8_t* m_scales;
  void* v;
  uint8_t* v_scales;
  float* master;
  const float* lr_ptr;
  const int32_t* step_ptr;
  const float* grad_scale;
  double lr, decay, log_b1, log_b2;  // for a step or a rate that is on the device
  float b1, not_b1, b2, not_b2, eps;
  float keep, rate, root;            // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t seed, step;
  int32_t count;
  uint32_t first[kListed];           // first chunk of each tensor
  uint32_t chunks;
  int32_t passes;
  Listed t[kListed];
};
static_assert(sizeof(AdamArgs) <= 4096, "kernel arguments");

__host__ __device__ inline uint32_t mix32(uint32_t h) {
  h = (h ^ (h >> 16)) * 0x6A09E667u;  // odd fractions of the square roots of 2 and 3
  h = (h ^ (h >> 15)) * 0xBB67AE85u;
  return h ^ (h >> 16);
}

__device__ __forceinline__ float bits_f32(uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ uint32_t f32_bits(float f) { return __builtin_bit_cast(uint32_t, f); }

// Eight values of a tensor, four from place i and four from place i + FAR on: next to each other (FAR 4) where
// blocks of 32 have to lie in four lanes, a workgroup's width apart where every access shall cover whole lines with
// 4 bytes a value. As they were read: fp32, or bf16 in the first half of lo (FAR 4: all of lo, or of lo and hi).
struct Eight {
  u32x4 lo, hi;
};

template <class V>
__device__ __forceinline__ V stream_in(const void* p) {
  return __builtin_nontemporal_load(static_cast<const V*>(p));
}
template <class V>
__device__ __forceinline__ void stream_out(void* p, V v) {
  __builtin_nontemporal_store(v, static_cast<V*>(p));
}

// Where not all of the chunk's values are there, or not aligned, they are read one by one as fp32, zeros from n on.
template <int FAR>
__device__ __forceinline__ Eight read_values(const void* base, bool f32, bool whole, int64_t i, int64_t n) {
  Eight x = {};
  if (whole) {
    if (f32) {
      const float* p = static_cast<const float*>(base) + i;
      if constexpr (FAR == 4) {  // (half lines: past the caches they would be fetched twice)
        x.lo = reinterpret_cast<const u32x4*>(p)[0], x.hi = reinterpret_cast<const u32x4*>(p)[1];
      } else {
        x.lo = stream_in<u32x4>(p), x.hi = stream_in<u32x4>(p + FAR);
      }
    } else {
      const uint16_t* p = static_cast<const uint16_t*>(base) + i;
      if constexpr (FAR == 4) {
        x.lo = stream_in<u32x4>(p);
      } else {
        const u32x2_t a = stream_in<u32x2_t>(p), b = stream_in<u32x2_t>(p + FAR);
        x.lo = u32x4{a[0], a[1], b[0], b[1]};
      }
    }
    return x;
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int64_t k = i + (j < 4 ? j : FAR + j - 4);
    uint32_t b = 0;
    if (k < n)
      b = f32 ? static_cast<const uint32_t*>(base)[k] : (uint32_t)static_cast<const uint16_t*>(base)[k] << 16;
    if (j < 4) x.lo[j] = b;
    else x.hi[j - 4] = b;
  }
  return x;
}

__device__ __forceinline__ void widen(const Eight& e, bool f32, float (&x)[kPer]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (f32) {
      x[j] = bits_f32(e.lo[j]), x[4 + j] = bits_f32(e.hi[j]);
    } else {
      x[2 * j] = bits_f32(e.lo[j] << 16), x[2 * j + 1] = bits_f32(e.lo[j] & 0xFFFF0000u);
    }
  }
}

// The largest magnitude of eight values; a NaN if one is.
__device__ __forceinline__ float largest(const float (&x)[kPer]) {
  float top = __builtin_fabsf(x[0]);
#pragma unroll
  for (int j = 1; j < kPer; ++j) top = __builtin_elementwise_maximum(top, __builtin_fabsf(x[j]));
  return top;
}

// bf16 of eight values, each with its dropped half added to 16 random bits: it rounds up with the probability of
// what it drops. What is not finite rounds as usual.
__device__ __forceinline__ u32x4 random_bf16(const float (&x)[kPer], const uint32_t (&r)[kPer]) {
  u32x4 o;
  if (largest(x) < __builtin_inff()) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = __builtin_amdgcn_perm(f32_bits(x[2 * j + 1]) + (r[2 * j + 1] & 0xFFFFu),
                                   f32_bits(x[2 * j]) + (r[2 * j] & 0xFFFFu), 0x07060302u);
    return o;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t h[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float v = x[2 * j + k];
      h[k] = __builtin_fabsf(v) < __builtin_inff() ? (f32_bits(v) + (r[2 * j + k] & 0xFFFFu)) >> 16 : f32_to_bf16_bits(v);
    }
    o[j] = h[0] | h[1] << 16;
  }
  return o;
}

template <bool RANDOM, int FAR>
__device__ __forceinline__ void store_values(void* base, bool f32, bool whole, int64_t i, int64_t n,
                                             const float (&x)[kPer], const uint32_t (&r)[kPer]) {
  if (f32) {
    float* p = static_cast<float*>(base) + i;
    if (whole) {
      const f32x4_t lo = {x[0], x[1], x[2], x[3]}, hi = {x[4], x[5], x[6], x[7]};
      if constexpr (FAR == 4) {  // (half lines: past the caches they would be written twice)
        reinterpret_cast<f32x4_t*>(p)[0] = lo;
        reinterpret_cast<f32x4_t*>(p)[1] = hi;
      } else {
        stream_out(p, lo);
        stream_out(p + FAR, hi);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int k = j < 4 ? j : FAR + j - 4;
        if (i + k < n) p[k] = x[j];
      }
    }
    return;
  }
  u32x4 o;
  if constexpr (RANDOM) {
    o = random_bf16(x, r);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
  }
  uint16_t* p = static_cast<uint16_t*>(base) + i;
  if (whole) {
    if constexpr (FAR == 4) {
      stream_out(p, o);
    } else {
      stream_out(p, u32x2_t{o[0], o[1]});
      stream_out(p + FAR, u32x2_t{o[2], o[3]});
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int k = j < 4 ? j : FAR + j - 4;
      if (i + k < n) p[k] = (uint16_t)(o[j >> 1] >> (16 * (j & 1)));
    }
  }
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xF, 0xF, true);
  return x > y ? x : y;
}

// The largest magnitude of a block, as bits (a NaN's above all), in each of the four lanes that hold it.
__device__ __forceinline__ uint32_t block_max(const float (&x)[kPer]) {
  return dpp_max<0x4E>(dpp_max<0xB1>(f32_bits(largest(x)) & 0x7FFFFFFFu));
}

// The scale byte for a block's largest magnitude, `up` powers of two below it, at least 1.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, uint32_t up) {
  const uint32_t field = top >> 23;
  return field == 255 ? 255u : (field > up ? field - up : 1u);
}

__device__ __forceinline__ void decode_m(u32x2_t q, uint32_t s, float (&x)[kPer]) {
  const float scale = bits_f32(s << 23);  // byte 255: an infinity, which makes NaN of the zero codes
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[h], true);
    x[4 * h] = lo[0] * scale, x[4 * h + 1] = lo[1] * scale, x[4 * h + 2] = hi[0] * scale, x[4 * h + 3] = hi[1] * scale;
  }
}

__device__ __forceinline__ uint32_t encode_m(const float (&x)[kPer], u32x2_t& q) {
  const uint32_t s = scale_byte(block_max(x), 7);
  const float inverse = bits_f32((254u - (s == 255 ? 254u : s)) << 23);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h] * inverse, x[4 * h + 1] * inverse, 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2] * inverse, x[4 * h + 3] * inverse, c, true);
    q[h] = s == 255 ? 0u : (uint32_t)c;
  }
  return s;
}

__device__ __forceinline__ void decode_v(u32x2_t q, uint32_t s, float (&x)[kPer]) {
  const uint32_t scale = s << 23, nothing = s == 255 ? 0x7FC00000u : 0u;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const uint32_t c = (q[j >> 2] >> (8 * (j & 3))) & 0xFFu;
    x[j] = bits_f32(c == 0 ? nothing : (c << 20) + scale);  // (a block of byte 255 has zero codes)
  }
}

template <bool RANDOM>
__device__ __forceinline__ uint32_t encode_v(const float (&x)[kPer], const uint32_t (&r)[kPer], u32x2_t& q) {
  const uint32_t s = scale_byte(block_max(x), 30);
  q = u32x2_t{0u, 0u};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int32_t b = (int32_t)f32_bits(x[j]);
    int32_t c = b - (int32_t)(s << 23);
    if constexpr (RANDOM) c += (int32_t)((r[j] >> 16) << 4);
    else c += 0x7FFFF + ((b >> 20) & 1);
    c >>= 20;
    // the middle one of c, 1 and b: at least 1, and 0 for b = 0, whose c is negative
    c = max(min(c, max(1, b)), min(1, b));
    q[j >> 2] |= (uint32_t)c << (8 * (j & 3));
  }
  if (s == 255) q = u32x2_t{0u, 0u};
  return s;
}

// What a thread holds of a pass before its step.
template <bool Q8>
struct Held {
  Eight grad, param;
  Eight m, v;  // fp32 moments, or codes in the first two words
  uint32_t m_scale, v_scale;
};

// A chunk's tensor and place.
struct Where {
  Listed t;
  int64_t base;
  bool whole, p_whole, g_whole;  // all of the chunk's values are there; and aligned
};

// A pass is 8 values a thread; with 8-bit moments they are consecutive, and since a tensor's moments begin at a
// multiple of 32, a block of 32 lies in four neighbouring lanes. A pass's loads go out before the step of the one
// before it.
// PRECISE: root and quotient as the compiler's own; otherwise the instructions themselves, each within an ulp
// but a second moment below 2^-126 counts as 0, which an eps from kLeastEps on hides (2^-63 / sqrt(1 - b2^t) of it).
template <bool Q8, bool MASTER, bool RANDOM, bool PRECISE>
__global__ __launch_bounds__(kThreads) void adamw_kernel(const AdamArgs g) {
  const int lane = threadIdx.x & 63;
  float keep = g.keep, rate = g.rate, root = g.root, gs = 1.0f;
  uint32_t step = g.step;
  if (g.lr_ptr != nullptr || g.step_ptr != nullptr) {
    const double lr = g.lr_ptr != nullptr ? (double)*g.lr_ptr : g.lr;
    const int32_t t = g.step_ptr != nullptr ? *g.step_ptr : (int32_t)g.step;
    step = (uint32_t)(t < 1 ? 1 : t);
    keep = (float)(1.0 - lr * g.decay);
    rate = (float)(lr / -expm1(step * g.log_b1));
    root = (float)(1.0 / sqrt(-expm1(step * g.log_b2)));
  }
  if (g.grad_scale != nullptr) gs = *g.grad_scale;
  const uint32_t key = mix32(g.seed ^ mix32(step));
  // first chunks of the tensors, for the search
  const uint32_t first0 = lane < g.count ? g.first[lane] : ~0u;
  const uint32_t first1 = 64 + lane < g.count ? g.first[lane + 64 < kListed ? lane + 64 : 0] : ~0u;

  auto find = [&](uint32_t chunk) {
    const int e = __builtin_amdgcn_readfirstlane(__popcll(__ballot(first0 <= chunk)) + __popcll(__ballot(first1 <= chunk))) - 1;
    Where w;
    w.t = g.t[e];
    w.base = (int64_t)(chunk - g.first[e]) * (g.passes * kPass);
    w.whole = w.base + g.passes * kPass <= w.t.n;
    w.p_whole = w.whole && (w.t.flags & kParamAligned), w.g_whole = w.whole && (w.t.flags & kGradAligned);
    return w;
  };
  constexpr int kFar = Q8 ? 4 : 4 * kThreads;
  auto place_of = [&](const Where& w, int pass) {
    return w.base + pass * kPass + (int64_t)threadIdx.x * (Q8 ? kPer : 4);
  };
  // whole blocks: what lies behind a tensor's last value, up to a multiple of 32, is held at zero
  auto held = [&](const Where& w) { return (w.t.n + 31) & ~(int64_t)31; };

  auto read = [&](Held<Q8>& h, const Where& w, int pass) {
    const int64_t i = place_of(w, pass), at = w.t.at + i;
    if (!w.whole && i >= held(w)) return;
    h.grad = read_values<kFar>(w.t.grad, w.t.flags & kGradF32, w.g_whole, i, w.t.n);
    if constexpr (MASTER) h.param = read_values<kFar>(g.master + w.t.at, true, w.whole, i, held(w));
    else h.param = read_values<kFar>(w.t.param, w.t.flags & kParamF32, w.p_whole, i, w.t.n);
    if constexpr (Q8) {
      const u32x2_t mq = stream_in<u32x2_t>(static_cast<const uint8_t*>(g.m) + at);
      const u32x2_t vq = stream_in<u32x2_t>(static_cast<const uint8_t*>(g.v) + at);
      h.m.lo[0] = mq[0], h.m.lo[1] = mq[1], h.v.lo[0] = vq[0], h.v.lo[1] = vq[1];
      h.m_scale = g.m_scales[at >> 5], h.v_scale = g.v_scales[at >> 5];
    } else {
      h.m = read_values<kFar>(static_cast<const float*>(g.m) + w.t.at, true, w.whole, i, held(w));
      h.v = read_values<kFar>(static_cast<const float*>(g.v) + w.t.at, true, w.whole, i, held(w));
    }
  };

  auto update = [&](const Held<Q8>& h, const Where& w, int pass) {
    const int64_t i = place_of(w, pass), at = w.t.at + i;
    if (!w.whole && i >= held(w)) return;
    float gr[kPer], p[kPer], m[kPer], v[kPer];
    uint32_t r[kPer];
    widen(h.grad, !w.g_whole || (w.t.flags & kGradF32), gr);
    widen(h.param, MASTER || !w.p_whole || (w.t.flags & kParamF32), p);
    if constexpr (Q8) {
      decode_m(u32x2_t{h.m.lo[0], h.m.lo[1]}, h.m_scale, m);
      decode_v(u32x2_t{h.v.lo[0], h.v.lo[1]}, h.v_scale, v);
    } else {
      widen(h.m, true, m);
      widen(h.v, true, v);
    }
    // (the places of four values share their upper half: they begin at a multiple of 4)
    uint32_t place[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t from = (uint64_t)at + k * kFar;
      place[k] = (uint32_t)from + (uint32_t)(from >> 32) * 0x9E3779B1u + key;
    }
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const float x = gr[j] * gs;
      m[j] = m[j] * g.b1 + x * g.not_b1;
      v[j] = v[j] * g.b2 + (x * x) * g.not_b2;
      float step_of;
      if constexpr (PRECISE) step_of = m[j] / (sqrtf(v[j]) * root + g.eps);
      else step_of = m[j] * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_sqrtf(v[j]), root, g.eps));
      p[j] = p[j] * keep - step_of * rate;
      if constexpr (RANDOM) r[j] = mix32(place[j >> 2] + (j & 3));
    }
    if (!w.whole) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (i + (j < 4 ? j : kFar + j - 4) >= w.t.n) m[j] = v[j] = p[j] = 0.0f;
    }
    store_values<RANDOM && !MASTER, kFar>(w.t.param, w.t.flags & kParamF32, w.p_whole, i, w.t.n, p, r);
    if constexpr (MASTER) store_values<false, kFar>(g.master + w.t.at, true, w.whole, i, held(w), p, r);
    if constexpr (Q8) {
      u32x2_t mq, vq;
      const uint32_t ms = encode_m(m, mq), vs = encode_v<RANDOM>(v, r, vq);
      stream_out(static_cast<uint8_t*>(g.m) + at, mq);
      stream_out(static_cast<uint8_t*>(g.v) + at, vq);
      if ((threadIdx.x & 3) == 0) {
        g.m_scales[at >> 5] = (uint8_t)ms;
        g.v_scales[at >> 5] = (uint8_t)vs;
      }
    } else {
      store_values<false, kFar>(static_cast<float*>(g.m) + w.t.at, true, w.whole, i, held(w), m, r);
      store_values<false, kFar>(static_cast<float*>(g.v) + w.t.at, true, w.whole, i, held(w), v, r);
    }
  };

  const bool two = g.passes == 2;
  uint32_t chunk = blockIdx.x;
  if (chunk >= g.chunks) return;
  Where here = find(chunk);
  Held<Q8> first = {}, second = {};
  read(first, here, 0);
  for (;;) {
    if (two) read(second, here, 1);
    update(first, here, 0);
    chunk += gridDim.x;
    if (chunk >= g.chunks) break;
    const Where next = find(chunk);
    read(first, next, 0);
    if (two) update(second, here, 1);
    here = next;
  }
  if (two) update(second, here, 1);
}

// The values of 8-bit moments as bf16 (exact: three bits of mantissa), 8 a thread.
__global__ __launch_bounds__(kThreads) void moments_kernel(const uint8_t* __restrict__ m, const uint8_t* __restrict__ ms,
                                                           const uint8_t* __restrict__ v, const uint8_t* __restrict__ vs,
                                                           int64_t n, uint16_t* __restrict__ m_out,
                                                           uint16_t* __restrict__ v_out) {
  const int64_t step = (int64_t)gridDim.x * kThreads * kPer;
  for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * kPer; i < n; i += step) {
    float x[kPer];
    u32x4 o;
    decode_m(*reinterpret_cast<const u32x2_t*>(m + i), ms[i >> 5], x);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<u32x4*>(m_out + i) = o;
    decode_v(*reinterpret_cast<const u32x2_t*>(v + i), vs[i >> 5], x);
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<u32x4*>(v_out + i) = o;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

hipError_t launch_adamw(const moe_adamw_tensor* list, void* const* params, const void* const* grads, int32_t count,
                        bool q8, void* m, uint8_t* m_scales, void* v, uint8_t* v_scales, float* master,
                        const moe_adamw_hyper& h, const float* lr_ptr, const int32_t* step_ptr, const float* grad_scale,
                        hipStream_t stream) {
  AdamArgs g;
  g.m = m, g.m_scales = m_scales, g.v = v, g.v_scales = v_scales, g.master = master;
  g.lr_ptr = lr_ptr, g.step_ptr = step_ptr, g.grad_scale = grad_scale;
  g.lr = h.lr, g.decay = h.weight_decay, g.log_b1 = std::log(h.beta1), g.log_b2 = std::log(h.beta2);
  g.b1 = (float)h.beta1, g.not_b1 = (float)(1.0 - h.beta1), g.b2 = (float)h.beta2, g.not_b2 = (float)(1.0 - h.beta2);
  g.eps = (float)h.eps;
  g.keep = (float)(1.0 - h.lr * h.weight_decay);
  g.rate = (float)(h.lr / -std::expm1(h.step * g.log_b1));
  g.root = (float)(1.0 / std::sqrt(-std::expm1(h.step * g.log_b2)));
  g.seed = h.seed, g.step = (uint32_t)h.step;
  const int64_t most = (int64_t)device_cu_count(current_device()) * 8;
  // Two passes a chunk hide the loads behind the steps; with too few chunks for that, one spreads the work over more
  // CUs (268 K values, fp32 throughout: 5.5 us, two 7.4; 398 M values: 2332 us, two 2174).
  int64_t values = 0;
  for (int32_t i = 0; i < count; ++i) values += list[i].n;
  g.passes = values < 2 * most * kPass ? 1 : 2;
  const int64_t per_chunk = g.passes * kPass;
  int32_t i = 0;
  while (i < count) {
    // as many tensors as the table holds and whose chunks a launch can count
    int64_t chunks = 0;
    g.count = 0;
    for (; i < count && g.count < kListed; ++i) {
      const int64_t n = (list[i].n + per_chunk - 1) / per_chunk;
      if (n == 0) continue;
      if (chunks + n > INT32_MAX) break;
      Listed& t = g.t[g.count];
      t.param = params[i], t.grad = grads[i], t.n = list[i].n, t.at = list[i].offset, t.pad = 0;
      t.flags = (list[i].param_dtype == MOE_F32 ? kParamF32 : 0) | (list[i].grad_dtype == MOE_F32 ? kGradF32 : 0) |
                (aligned16(t.param) ? kParamAligned : 0) | (aligned16(t.grad) ? kGradAligned : 0);
      g.first[g.count++] = (uint32_t)chunks;
      chunks += n;
    }
    if (g.count == 0) break;
    g.chunks = (uint32_t)chunks;
    const dim3 grid((unsigned)(chunks < most ? chunks : most)), block(kThreads);
    const bool random = h.stochastic != 0, precise = !q8 || h.eps < kLeastEps;
    auto run = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, block, 0, stream, g); };
    if (master != nullptr) {
      if (!q8) run(adamw_kernel<false, true, false, true>);  // (nothing left to round at random)
      else if (random) precise ? run(adamw_kernel<true, true, true, true>) : run(adamw_kernel<true, true, true, false>);
      else precise ? run(adamw_kernel<true, true, false, true>) : run(adamw_kernel<true, true, false, false>);
    } else if (q8) {
      if (random) precise ? run(adamw_kernel<true, false, true, true>) : run(adamw_kernel<true, false, true, false>);
      else precise ? run(adamw_kernel<true, false, false, true>) : run(adamw_kernel<true, false, false, false>);
    } else {
      random ? run(adamw_kernel<false, false, true, true>) : run(adamw_kernel<false, false, false, true>);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_adamw_moments(const uint8_t* m, const uint8_t* ms, const uint8_t* v, const uint8_t* vs, int64_t n,
                                uint16_t* m_out, uint16_t* v_out, hipStream_t stream) {
  if (n == 0) return hipSuccess;
  int64_t blocks = (n / kPer + kThreads - 1) / kThreads;
  const int64_t most = (int64_t)device_cu_count(current_device()) * 16;
  hipLaunchKernelGGL(moments_kernel, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, stream, m, ms, v,
                     vs, n, m_out, v_out);
  return hipGetLastError();
}

}  // namespace moe
