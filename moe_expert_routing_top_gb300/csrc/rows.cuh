// rows.cuh -- rows of fp32, bf16 or fp16 values by eight neighbouring columns a
// thread: loads, stores and e4m3 rounding shared by the norm, the gated
// activation and the combination of the experts' rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace moer {

// Eight neighbouring values as they lie in memory (16 bytes, fp32: 32).
template <typename T>
struct Raw8 {
  T v[8];
};

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
  else return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x) {
  if constexpr (sizeof(T) == 4) return x;
  else if constexpr (std::is_same<T, __half>::value) return __float2half_rn(x);
  else return __float2bfloat16_rn(x);
}

// n: columns left in the row from p on (may be <= 0: zeros).  VEC: the row's columns are a multiple
// of eight and every row starts on 16 bytes, so the eight are there or none is.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n) {
  Raw8<T> r;
  if constexpr (VEC) {
    constexpr int Q = sizeof(T) / 2;
    uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < Q; ++i) d[i] = n > 0 ? __ldg(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  return r;
}

// The same without the read-only path: for buffers that the call also writes.
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load8_rw(const T* p, int n) {
  Raw8<T> r;
  if constexpr (VEC) {
    constexpr int Q = sizeof(T) / 2;
    uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
    for (int i = 0; i < Q; ++i) d[i] = n > 0 ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.v[i] = i < n ? p[i] : from_f32<T>(0.f);
  }
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, const Raw8<T>& r, int n) {
  if constexpr (VEC) {
    constexpr int Q = sizeof(T) / 2;
    const uint4* s = reinterpret_cast<const uint4*>(&r);
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < Q; ++i) reinterpret_cast<uint4*>(p)[i] = s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = r.v[i];
  }
}

template <typename T>
__device__ __forceinline__ Raw8<T> pack8(const float (&f)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r.v[i] = from_f32<T>(f[i]);
  return r;
}

constexpr float E4M3_MAX = 448.f;
constexpr float QUANT_LEAST = 1e-30f;  // keeps a block of zeros' scale, and its reciprocal, finite

// Two values a / s rounded to nearest, from r = 1 / s rounded to nearest: the product and one correction by its
// exact residual (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990),
// with its sign turned twice, so that -0 stays -0.  Two lanes an instruction: one by one, the
// activation of 270,208 rows of 768 to 8 bits took 187 us instead of 180 (176 by the reciprocal alone).
__device__ __forceinline__ float2 quotients(float a0, float a1, float s, float r) {
  float2 q;
  asm("{\n\t.reg .b64 a, n, s, r, q, e;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 n, {%4, %5};\n\tmov.b64 s, {%6, %6};\n\tmov.b64 r, {%7, %7};\n\t"
      "mul.rn.f32x2 q, a, r;\n\tfma.rn.f32x2 e, q, s, n;\n\tmov.b64 s, {%8, %8};\n\tfma.rn.f32x2 q, e, s, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
      : "=f"(q.x), "=f"(q.y)
      : "f"(a0), "f"(a1), "f"(-a0), "f"(-a1), "f"(s), "f"(r), "f"(-r));
  return q;
}

// A block of 128 columns lies with 16 neighbouring lanes, eight each: stores their e4m3 values and
// the block's scale.  Warp-collective; n: columns left from the lane's first on.  The values are the
// fp32 quotients by the stored scale, rounded: by the reciprocal alone a value on the border between two
// codes can go to the farther one (one in a million of random rows).
template <bool VEC>
__device__ __forceinline__ void store_e4m3(const float (&y)[8], uint8_t* q, float* scale, int lane, int n) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(y[i]));  // fmaxf passes over a NaN
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL, m, d));
  const float s = fmaxf(m, QUANT_LEAST) * (1.f / E4M3_MAX);
  const float r = 1.f / s, c = r > 0.f ? s : 0.f;  // of an infinite scale: no correction, so that numbers give 0 and not NaN
  if (n <= 0) return;
  if ((lane & 15) == 0) *scale = s;
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __nv_cvt_float2_to_fp8x2(quotients(y[4 * h], y[4 * h + 1], c, r), __NV_SATFINITE, __NV_E4M3);
    const uint32_t b = __nv_cvt_float2_to_fp8x2(quotients(y[4 * h + 2], y[4 * h + 3], c, r), __NV_SATFINITE, __NV_E4M3);
    w[h] = a | (b << 16);
  }
  if constexpr (VEC) {
    *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
  }
}

}  // namespace moer
