// Element functions shared by the product epilogues (GEMM, GEMV), their
// gradient and the layer norm: typed loads and stores of rows that are bf16 or
// fp32, the activations with their derivatives, and the maximum of stored
// magnitudes.
//
// Activations, evaluated in fp32 (relative error below 2^-20; the 2-ulp
// ex2 / rcp / fast-divide forms, since an output is rounded to 2^-9 or
// compared at 2^-20, not at 2^-24):
//   relu       max(v, 0); a NaN stays a NaN
//   gelu       v Phi(v) = max(v, 0) - |v| g with g = erfc(|v| / sqrt 2) / 2, so
//              the negative tail keeps its relative accuracy (1 + erf cancels)
//   gelu_tanh  v/2 (1 + tanh u) = v / (1 + e^{-2u}), u = sqrt(2/pi) (v + 0.044715 v^3)
//   silu       v / (1 + e^{-v})
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "nvfp4.h"

namespace nvfp4 {

constexpr float kGeluC2 = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// g = erfc(a / sqrt 2) / 2 = e^{-a^2 / 2} t Q(t) / 2, t = 1 / (1 + 0.425 a /
// sqrt 2), for a >= 0; also e = e^{-a^2 / 2}.  Q: polynomial of degree 7 fitted
// to e^{x^2} erfc(x) / t for 0 <= x <= 9.3 with the least largest relative
// error (1.1e-7; 4e-7 with its evaluation in fp32): a GEMM with this gelu at
// K = 1024, where its epilogue is what takes the time, runs 2.1 times as fast as
// with erfcf (78 against 162 us, 4096 x 8192).  Past a = 16, e is 0.
__device__ __forceinline__ float normal_tail(float a, float& e) {
  const float t = __fdividef(1.0f, fmaf(0.3005203820f, a, 1.0f));
  float q = 0.0724736005f;
  q = fmaf(q, t, -0.3173076808f);
  q = fmaf(q, t, 0.4147784114f);
  q = fmaf(q, t, -0.1098528951f);
  q = fmaf(q, t, 0.2585873306f);
  q = fmaf(q, t, 0.1996419132f);
  q = fmaf(q, t, 0.2420118004f);
  q = fmaf(q, t, 0.2396674007f);
  e = __expf(-0.5f * a * a);
  return 0.5f * e * (t * q);
}

__device__ __forceinline__ float act_value(float v, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return v < 0.0f ? 0.0f : v;
    case NVFP4_ACT_GELU: {
      float e;
      const float a = fminf(fabsf(v), 16.0f);
      return (v < 0.0f ? 0.0f : v) - a * normal_tail(a, e);          // a NaN stays one
    }
    case NVFP4_ACT_GELU_TANH: return __fdividef(v, 1.0f + __expf(-kGeluC2 * v * fmaf(kGeluA * v, v, 1.0f)));
    case NVFP4_ACT_SILU: return __fdividef(v, 1.0f + __expf(-v));
    default: return v;
  }
}

// The same for an array, with one branch on the activation.
template <int N>
__device__ __forceinline__ void act_values(float (&x)[N], int act) {
  switch (act) {
    case NVFP4_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = act_value(x[i], NVFP4_ACT_RELU);
      break;
    case NVFP4_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = act_value(x[i], NVFP4_ACT_GELU);
      break;
    case NVFP4_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = act_value(x[i], NVFP4_ACT_GELU_TANH);
      break;
    case NVFP4_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) x[i] = act_value(x[i], NVFP4_ACT_SILU);
      break;
    default: break;
  }
}

// act'(v).  The logistic forms are written on e = e^{-|.|} <= 1, so neither
// p (1 - p) nor the tails cancel or overflow; past |v| = 16 (gelu) or 128
// (silu) the second term is below the smallest normal number and left out, so
// an infinite v gives the limit (0 or 1) instead of inf * 0.
__device__ __forceinline__ float act_slope(float v, int act) {
  switch (act) {
    case NVFP4_ACT_RELU: return v > 0.0f ? 1.0f : (v <= 0.0f ? 0.0f : v);
    case NVFP4_ACT_GELU: {
      float e;
      const float a = fminf(fabsf(v), 16.0f);
      const float g = normal_tail(a, e);
      const float p = v < 0.0f ? g : 1.0f - g;
      return v == v ? fmaf(kInvSqrt2Pi * e, copysignf(a, v), p) : v;
    }
    case NVFP4_ACT_GELU_TANH: {
      const float v2 = v * v;
      const float u2 = kGeluC2 * v * fmaf(kGeluA, v2, 1.0f);
      const float e = __expf(-fabsf(u2));
      const float r = __fdividef(1.0f, 1.0f + e);
      const float q = e * r;
      const float p = v < 0.0f ? q : r;
      return fabsf(v) < 16.0f ? fmaf(kGeluC2 * v * (q * r), fmaf(3.0f * kGeluA, v2, 1.0f), p) : (v == v ? p : v);
    }
    case NVFP4_ACT_SILU: {
      const float e = __expf(-fabsf(v));
      const float r = __fdividef(1.0f, 1.0f + e);
      const float q = e * r;
      const float p = v < 0.0f ? q : r;
      return fabsf(v) < 128.0f ? fmaf(v, q * r, p) : (v == v ? p : v);
    }
    default: return 1.0f;
  }
}

// Typed element access (T: __nv_bfloat16 or float).
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Magnitude of a stored value as fp32 bits: the unsigned order of these is the
// order of |v|, infinities and then NaNs last.
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t mag_bits(__nv_bfloat16 v) {
  return static_cast<uint32_t>(__bfloat16_as_ushort(v) & 0x7FFFu) << 16;
}

// One element of a bf16 or fp32 vector (a bias, a norm's weight).
__device__ __forceinline__ float load_param(const void* p, int f32, int64_t i) {
  return f32 ? __ldg(static_cast<const float*>(p) + i)
             : __bfloat162float(__ushort_as_bfloat16(__ldg(static_cast<const unsigned short*>(p) + i)));
}

}  // namespace nvfp4
