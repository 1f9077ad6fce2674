// Element functions shared by the product epilogues (GEMM, GEMV), their
// gradient and the layer norm: typed loads and stores of rows that are bf16 or
// fp32, the activations with their derivatives, and the maximum of stored
// magnitudes.
//
// Activations, evaluated in fp32 with the 2-ulp ex2 and rcp.  The rounding of an
// exponential's argument w moves e^w by |w| roundings, so the relative error is
// at most (8 + 2 X) 2^-23 with X the size of that argument (v^2 for gelu, 2 u for
// gelu_tanh, v for silu).  Emulated with correctly rounded ex2 and rcp: about
// 2^-20 for v > -2; in the negative tails, whose values are small against v,
// 2^-17.7 (gelu) and 2^-16.1 (gelu_tanh) at v = -10 and 2^-18 (silu) at v = -87.
// Outputs in bf16 are rounded to 2^-9, so only fp32 ones show it.  A logistic or
// a tail below 2^-126 is 0: silu is from v = -87.4 down.
//   relu       max(v, 0); a NaN stays a NaN
//   gelu       v Phi(v) = max(v, 0) - |v| g with g = erfc(|v| / sqrt 2) / 2, so
//              the negative tail keeps its relative accuracy (1 + erf cancels)
//   gelu_tanh  v/2 (1 + tanh u) = v / (1 + e^{-2u}), u = sqrt(2/pi) (v + 0.044715 v^3)
//   silu       v / (1 + e^{-v})
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "nvfp4.h"

namespace nvfp4 {

// Two fp32 lanes per instruction (add / mul / fma.rn.f32x2): these kernels are
// bound by instruction issue as much as by memory.
__device__ __forceinline__ unsigned long long bits2(float2 a) { return *reinterpret_cast<unsigned long long*>(&a); }
__device__ __forceinline__ float2 pair2(unsigned long long b) { return *reinterpret_cast<float2*>(&b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return pair2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
  return pair2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return pair2(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 2^x and 1 / x to 2 ulps (results below 2^-126 are 0), and the minimum and
// maximum that keep a NaN.
__device__ __forceinline__ float2 exp2_2(float2 x) {
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  return x;
}
__device__ __forceinline__ float2 rcp2(float2 x) {
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.x));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(x.y));
  return x;
}
__device__ __forceinline__ float2 min2(float2 x, float c) {
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(c));
  asm("min.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(c));
  return x;
}
__device__ __forceinline__ float2 max2(float2 x, float c) {
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.x) : "f"(c));
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(x.y) : "f"(c));
  return x;
}
__device__ __forceinline__ float2 abs2(float2 x) { return make_float2(fabsf(x.x), fabsf(x.y)); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluC2 = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// g = erfc(a / sqrt 2) / 2 = e^{-a^2 / 2} t Q(t) / 2, t = 1 / (1 + 0.425 a /
// sqrt 2), for a >= 0; also e = e^{-a^2 / 2}.  Q: polynomial of degree 7 fitted
// to e^{x^2} erfc(x) / t for 0 <= x <= 9.3 with the least largest relative
// error (1.1e-7; 4e-7 with its evaluation in fp32), the half taken into its
// coefficients: a GEMM with this gelu at K = 1024, where its epilogue is what
// takes the time, ran 2.1 times as fast as with erfcf (78 against 162 us, 4096
// x 8192).  Past a = 16, e is 0.
__device__ __forceinline__ float2 normal_tail2(float2 a, float2& e) {
  const float2 t = rcp2(fma2(both(0.3005203820f), a, both(1.0f)));
  float2 q = both(0.5f * 0.0724736005f);
  q = fma2(q, t, both(0.5f * -0.3173076808f));
  q = fma2(q, t, both(0.5f * 0.4147784114f));
  q = fma2(q, t, both(0.5f * -0.1098528951f));
  q = fma2(q, t, both(0.5f * 0.2585873306f));
  q = fma2(q, t, both(0.5f * 0.1996419132f));
  q = fma2(q, t, both(0.5f * 0.2420118004f));
  q = fma2(q, t, both(0.5f * 0.2396674007f));
  e = exp2_2(mul2(mul2(a, both(-0.5f * kLog2e)), a));
  return mul2(e, mul2(t, q));
}

// act(v) of two values.  A NaN stays one; an infinite v gives the limit where
// that is finite or v, except silu and gelu_tanh at -infinity (NaN, as
// v / (1 + e^{-v}) has there).
template <int kAct>
__device__ __forceinline__ float2 act_pair(float2 v) {
  if constexpr (kAct == NVFP4_ACT_RELU) {
    return max2(v, 0.0f);
  } else if constexpr (kAct == NVFP4_ACT_GELU) {
    float2 e;
    const float2 a = min2(abs2(v), 16.0f);
    return fma2(both(-1.0f), mul2(a, normal_tail2(a, e)), max2(v, 0.0f));
  } else if constexpr (kAct == NVFP4_ACT_GELU_TANH) {
    const float2 m = mul2(v, both(-kGeluC2 * kLog2e));
    const float2 w = fma2(mul2(v, both(kGeluA)), v, both(1.0f));
    return mul2(v, rcp2(add2(exp2_2(mul2(m, w)), both(1.0f))));
  } else if constexpr (kAct == NVFP4_ACT_SILU) {
    return mul2(v, rcp2(add2(exp2_2(mul2(v, both(-kLog2e))), both(1.0f))));
  } else {
    return v;
  }
}

// act'(v) of two values.  The logistic forms are written on e = e^{-|.|} <= 1,
// so neither p (1 - p) nor the tails cancel or overflow, and on v held to the
// range outside which act' is 0 or 1 to the last bit (|v| <= 16, silu 128), so
// an infinite v gives the limit; a NaN stays one.
template <int kAct>
__device__ __forceinline__ float2 slope_pair(float2 v) {
  if constexpr (kAct == NVFP4_ACT_RELU) {
    const auto one = [](float x) { return x > 0.0f ? 1.0f : (x <= 0.0f ? 0.0f : x); };
    return make_float2(one(v.x), one(v.y));
  } else if constexpr (kAct == NVFP4_ACT_GELU) {
    float2 e;
    v = max2(min2(v, 16.0f), -16.0f);
    const float2 g = normal_tail2(abs2(v), e);
    const float2 p = make_float2(v.x < 0.0f ? g.x : 1.0f - g.x, v.y < 0.0f ? g.y : 1.0f - g.y);
    return fma2(mul2(e, both(kInvSqrt2Pi)), v, p);
  } else if constexpr (kAct == NVFP4_ACT_GELU_TANH || kAct == NVFP4_ACT_SILU) {
    constexpr bool kGelu = kAct == NVFP4_ACT_GELU_TANH;
    v = max2(min2(v, kGelu ? 16.0f : 128.0f), kGelu ? -16.0f : -128.0f);
    // logistic argument u = w v, slope p + v u'(v) p (1 - p)
    float2 u = v, du = v;                       // u, v u'(v)
    if constexpr (kGelu) {
      const float2 v2 = mul2(v, v), m = mul2(v, both(kGeluC2));
      u = mul2(m, fma2(v2, both(kGeluA), both(1.0f)));
      du = mul2(m, fma2(v2, both(3.0f * kGeluA), both(1.0f)));
    }
    const float2 e = exp2_2(mul2(abs2(u), both(-kLog2e)));
    const float2 r = rcp2(add2(e, both(1.0f))), q = mul2(e, r);
    const float2 p = make_float2(v.x < 0.0f ? q.x : r.x, v.y < 0.0f ? q.y : r.y);
    return fma2(du, mul2(q, r), p);
  } else {
    return both(1.0f);
  }
}

// Calls f with the activation as a compile-time constant.
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case NVFP4_ACT_RELU: f(std::integral_constant<int, NVFP4_ACT_RELU>{}); break;
    case NVFP4_ACT_GELU: f(std::integral_constant<int, NVFP4_ACT_GELU>{}); break;
    case NVFP4_ACT_GELU_TANH: f(std::integral_constant<int, NVFP4_ACT_GELU_TANH>{}); break;
    case NVFP4_ACT_SILU: f(std::integral_constant<int, NVFP4_ACT_SILU>{}); break;
    default: f(std::integral_constant<int, NVFP4_ACT_NONE>{}); break;
  }
}

template <int N>
__device__ __forceinline__ void act_values(float2 (&x)[N], int act) {
  with_act(act, [&](auto a) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = act_pair<decltype(a)::value>(x[i]);
  });
}

// A chunk: 8 elements as 4 pairs.
struct Chunk {
  float2 v[4];
  __device__ __forceinline__ float get(int e) const { return e & 1 ? v[e >> 1].y : v[e >> 1].x; }
};

__device__ __forceinline__ Chunk unpack_chunk(const uint4 w) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  Chunk c;
#pragma unroll
  for (int i = 0; i < 4; ++i) c.v[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
  return c;
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

// Stores a chunk rounded to T (unless out is null) and takes it into the running maximum of stored
// magnitudes (Mag: both halves of a word for bf16, where one instruction takes
// the larger magnitudes of two pairs and keeps a NaN).
template <typename T>
struct Mag {
  uint32_t m = 0;
  __device__ __forceinline__ void pair(uint32_t u) {
    asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(u));
  }
  __device__ __forceinline__ uint32_t bits() const {
    return max((m & 0x7FFFu) << 16, m & 0x7FFF0000u);
  }
};
template <>
struct Mag<float> {
  uint32_t m = 0;
  __device__ __forceinline__ uint32_t bits() const { return m; }
};

template <typename T>
__device__ __forceinline__ void store_chunk(T* out, const Chunk& x, Mag<T>& mag) {
  if constexpr (sizeof(T) == 2) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x.v[i].x, x.v[i].y);
      u[i] = *reinterpret_cast<const uint32_t*>(&h);
      mag.pair(u[i]);
    }
    if (out) *reinterpret_cast<uint4*>(out) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    if (out) {
      *reinterpret_cast<float4*>(out) = make_float4(x.v[0].x, x.v[0].y, x.v[1].x, x.v[1].y);
      *reinterpret_cast<float4*>(out + 4) = make_float4(x.v[2].x, x.v[2].y, x.v[3].x, x.v[3].y);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) mag.m = max(mag.m, mag_bits(x.get(e)));
  }
}

}  // namespace nvfp4
