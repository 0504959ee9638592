// score.cuh -- the scores of moer_score_topk and its gradient: logit types,
// the score functions and the parameters that their kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"
#include "rank.cuh"

namespace moer {

struct ScoreParams {
  const void* logits;
  int64_t T, ld_token, ld_layer;  // strides in elements
  int E, k, L;
  int score, renorm, n_group, top_group, group_best;
  float scale;
  int vec;             // 1: every row of logits (and gradients) takes 4-element vector access
  const float* bias;   // [L][E] or NULL
  uint8_t* topk;       // out [L][T][k]
  float* weights;      // out [L][T][k] or NULL
  float* partial;      // [units][E] score sums of each unit, or NULL
  int span, nspan;     // tokens of a unit, units of a layer
  int wide;            // 1: rows take 16-byte access (the fast kernel's blocks of 8 logits)
  int even;            // 2: k = 8, weights on 16 bytes; 1: k even, weights on 8 bytes; 0: neither
  // 2^8, known at run time only, so that a key's shift-and-insert stays one
  // multiply-add (FMA pipe) and off the integer ALU pipe that the networks fill
  uint32_t key_mul;
  // gradient
  const uint8_t* ids;        // [L][T][k]
  const float* d_weights;    // [L][T][k]
  const float* d_score_sum;  // [L][E] or NULL
  void* d_logits;
  int64_t ldg_token, ldg_layer;
  uint32_t* status;
};

// What the fast kernel's choice goes by.  A kernel for each keeps its code short:
// one for all that take scores or groups took as long with a fifth fewer instructions
// an expert, for it left the instruction cache between its branches.
enum ScoreKind {
  BY_LOGIT = 0,        // the logits alone; weights from the chosen ones
  SOFTMAX_SUMS = 1,    // the logits; with the column pass of a softmax
  SIGMOID_SUMS = 2,    // the logits; with the column pass of a sigmoid
  BY_GROUP = 3,        // the logits, in groups
  BY_SIGMOID = 4,      // scores with a bias
  BY_SOFTMAX = 5
};
inline ScoreKind score_kind(bool bias, int n_group, bool sums, bool soft, bool renorm) {
  if (bias) return soft ? BY_SOFTMAX : BY_SIGMOID;
  if (n_group > 1) return BY_GROUP;
  if (soft) return sums || !renorm ? SOFTMAX_SUMS : BY_LOGIT;
  return sums ? SIGMOID_SUMS : BY_LOGIT;
}
// Experts of the quads that a group of gs lies in, where it begins in the worst place.
__host__ __device__ constexpr int group_span(int gs) { return (gs + ((gs & 1) ? 3 : (gs & 2)) + 3) & ~3; }

// Blocks of 128 threads of the fast kernel on an SM, which sets its registers.  fp32
// choices by group or score with 4 blocks / 5 (which spill): 192 / 214 us by sigmoid with
// bias, 137 / 167 by logit, 26 x 20,000 rows of 256 in 8 groups; 122 / 161 us, 48 x 20,000
// rows of 128 in 4.  bf16 ones: 174 / 169 and 130 / 131 us.  The others with 4 / 5 / 6:
// 3.1 M rows x 128 fp32 341 / 291 / 334 us, 780 k x 64 bf16 with column pass 72 / 70 /
// 67 us.  A top 16 holds 8 keys more a lane.
constexpr int score_resident(int elem, int kind, int kt) {
  return kt > 8 || (elem == 4 && kind >= BY_GROUP) ? 4 : kind >= BY_GROUP ? 5 : elem == 2 ? 6 : 5;
}

constexpr float NEG_INF = -__builtin_huge_valf();
constexpr float LOWEST = -3.402823466e38f;  // the lowest finite number

// ------------------------------------------------------- four logits at once
// Logits are held as fp32 whatever their type (an exact conversion); a
// gradient is rounded once, to nearest even, when it is stored.
template <typename X>
struct Quad;
template <>
struct Quad<float> {
  using V = float4;
  __device__ static void get(const V& v, float (&x)[4]) { x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w; }
  __device__ static V put(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
  __device__ static float one(float v) { return v; }
  __device__ static float back(float v) { return v; }
};
template <>
struct Quad<__nv_bfloat16> {
  using V = uint2;
  __device__ static void get(const V& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  __device__ static V put(const float (&x)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  __device__ static float one(__nv_bfloat16 v) { return __bfloat162float(v); }
  __device__ static __nv_bfloat16 back(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Quad<__half> {
  using V = uint2;
  __device__ static void get(const V& v, float (&x)[4]) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  }
  __device__ static V put(const float (&x)[4]) {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  __device__ static float one(__half v) { return __half2float(v); }
  __device__ static __half back(float v) { return __float2half_rn(v); }
};

template <typename X>
__device__ __forceinline__ void load4(const X* p, bool vec, float (&x)[4]) {
  if (vec) {
    Quad<X>::get(*reinterpret_cast<const typename Quad<X>::V*>(p), x);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = Quad<X>::one(p[j]);
  }
}
template <typename X>
__device__ __forceinline__ void store4(X* p, bool vec, const float (&x)[4]) {
  if (vec) {
    *reinterpret_cast<typename Quad<X>::V*>(p) = Quad<X>::put(x);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = Quad<X>::back(x[j]);
  }
}

// Blocks of 8 logits as they are stored.
template <int EB>
struct Raw;
template <>
struct Raw<4> {
  float v[8];
  // room: experts left in the row; the block's others are `fill` (-inf or 0)
  template <typename X>
  __device__ __forceinline__ void load(const float* p, int room, bool, float fill = NEG_INF) {
    float4 a = make_float4(fill, fill, fill, fill), b = a;
    if (room >= 4) a = *reinterpret_cast<const float4*>(p);
    if (room >= 8) b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  // two quads apart, either of which may be missing
  template <typename X>
  __device__ __forceinline__ void load2(const float* p, bool has, const float* q, bool has2, float fill) {
    float4 a = make_float4(fill, fill, fill, fill), b = a;
    if (has) a = *reinterpret_cast<const float4*>(p);
    if (has2) b = *reinterpret_cast<const float4*>(q);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  template <typename X>
  __device__ __forceinline__ void get(float (&x)[8]) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j];
  }
};
template <>
struct Raw<2> {
  uint4 v;
  template <typename X>
  __device__ __forceinline__ void load(const X* p, int room, bool wide, float fill = NEG_INF) {
    const uint32_t low = fill == 0.f ? 0u : std::is_same<X, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    v = make_uint4(low, low, low, low);
    if (wide) {
      if (room >= 8) v = *reinterpret_cast<const uint4*>(p);
      else if (room >= 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        v.x = a.x, v.y = a.y;
      }
    } else {
      if (room >= 4) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        v.x = a.x, v.y = a.y;
      }
      if (room >= 8) {
        const uint2 a = *reinterpret_cast<const uint2*>(p + 4);
        v.z = a.x, v.w = a.y;
      }
    }
  }
  template <typename X>
  __device__ __forceinline__ void load2(const X* p, bool has, const X* q, bool has2, float fill) {
    const uint32_t low = fill == 0.f ? 0u : std::is_same<X, __half>::value ? 0xFC00FC00u : 0xFF80FF80u;
    v = make_uint4(low, low, low, low);
    if (has) {
      const uint2 a = *reinterpret_cast<const uint2*>(p);
      v.x = a.x, v.y = a.y;
    }
    if (has2) {
      const uint2 a = *reinterpret_cast<const uint2*>(q);
      v.z = a.x, v.w = a.y;
    }
  }
  template <typename X>
  __device__ __forceinline__ void get(float (&x)[8]) const {
    float a[4], b[4];
    Quad<X>::get(make_uint2(v.x, v.y), a);
    Quad<X>::get(make_uint2(v.z, v.w), b);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = a[j], x[4 + j] = b[j];
  }
};

// ------------------------------------------------------------------ scores
__device__ __forceinline__ float rcp_approx(float x) {  // within 1 ulp
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float ex2_approx(float x) {  // 2 units in the last place
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float fma_sat(float a, float b, float c) {  // NaN -> 0
  float r;
  asm("fma.rn.sat.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float mul_ftz(float a, float b) {  // numbers under the normal range are 0
  float r;
  asm("mul.rn.ftz.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// A logit that counts: -inf for a masked expert, NaN included.
__device__ __forceinline__ float live_logit(float x) { return x == x ? x : NEG_INF; }
// 1 / (1 + exp(-x)): 0 at -inf, 1 at +inf; below x = -87.3 the result is under
// the smallest normal number and is 0 (the reciprocal flushes it).
__device__ __forceinline__ float sigmoid(float x) { return rcp_approx(1.f + expf(-x)); }
// s (1 - s) without the cancellation of 1 - s: t / (1 + t)^2, t = exp(-|x|); 0 where s is.
__device__ __forceinline__ float sigmoid_slope(float x) {
  const float t = expf(-fabsf(x)), r = rcp_approx(1.f + t);
  return mul_ftz(t, r * r);
}
// exp(x - m) for x <= m, where m is the largest of a set: equal infinities
// give 1 (they share the weight), and a set without any expert gives 0.
__device__ __forceinline__ float exp_below(float x, float m) {
  if (x == NEG_INF) return 0.f;
  return x == m ? 1.f : expf(x - m);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// Whether n holds a logit exactly: 16-bit logits of size 2^-5 to 128 are
// multiples of 2^-15, a step of n, so that equal n mean equal logits there and
// the id in the key orders them.
template <int EB>
__device__ __forceinline__ bool exact_n(int n) {
  return EB == 2 && abs(n - 4194304) > 1024 && n > 0;
}

// Inverse of rank_key for keys of numbers (NaN's key 1 gives -inf: it adds
// nothing to a group).
__device__ __forceinline__ float rank_value(uint32_t key) {
  if (key <= 1u) return NEG_INF;
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7FFFFFFFu) : ~key);
}

}  // namespace moer
