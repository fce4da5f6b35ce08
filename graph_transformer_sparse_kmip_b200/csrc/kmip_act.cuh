// kmip_act.cuh -- activations of the group norm and the gated feed-forward
// block, and their derivatives.
//
// T is the element type that results are rounded to: for bf16 (half a step is
// 2^-9 to 2^-8 of the value) the exponential and the quotient are the approximate
// instructions, good to about 2^-21 together: four instructions a sigmoid,
// where the accurate ones made the feed-forward's epilogue twice as long as
// its products.  fp32 takes the accurate ones.
#pragma once

#include "kmip_common.cuh"

namespace kmip {

// 2^x and 1/x by one instruction each, subnormals as zero (2^x = 0 below
// -126, 1/inf = 0: both what the sigmoid needs).
__device__ __forceinline__ float ex2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (sizeof(T) == 2)
    return rcp_fast(1.f + ex2_fast(-1.4426950408889634f * z));  // log2(e)
  else
    return 1.f / (1.f + expf(-z));
}

// Phi(z) and phi(z), the normal distribution's.  fp32: erfc and exp.  bf16:
// Phi(-|z|) = t q(t) exp(-z^2 / 2) with t = 1 / (1 + p |z|) and q the polynomial
// of degree 6 (p chosen with it) whose largest relative error is least, fitted by
// linear programming to erfcx(|z| / sqrt 2) / 2: 2^-21, with the roundings 2^-18
// down to z = -9 and, as the exponent grows, 2^-17 to -13, where the result leaves
// the normal numbers.  So gelu keeps its digits in the tail, where a bound on the
// absolute error of erfc would not.  The exponential is phi's too.  (With erfc the
// group norm's backward took three times as long as with silu.)
template <typename T>
__device__ __forceinline__ void gauss(float z, float& cdf, float& pdf) {
  if constexpr (sizeof(T) == 2) {
    const float e = ex2_fast(-0.72134752044448170f * z * z);  // -log2(e) / 2
    const float t = rcp_fast(fmaf(0.2639416f, fabsf(z), 1.f));
    float q = fmaf(-0.069472544f, t, 0.2042903f);
    q = fmaf(q, t, -0.077432394f);
    q = fmaf(q, t, 0.1494758f);
    q = fmaf(q, t, 0.080134764f);
    q = fmaf(q, t, 0.107858144f);
    q = fmaf(q, t, 0.10514564f);
    const float tail = q * t * e;
    cdf = z < 0.f ? tail : 1.f - tail;
    pdf = 0.39894228040143268f * e;
  } else {
    cdf = 0.5f * erfcf(-0.70710678118654752f * z);
    pdf = 0.39894228040143268f * expf(-0.5f * z * z);
  }
}

// act(z).  relu passes a NaN on.
template <typename T, int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == KMIP_ACT_SILU) return z * sigmoid<T>(z);
  if constexpr (ACT == KMIP_ACT_GELU) {
    float c, d;
    gauss<T>(z, c, d);
    return z * c;
  }
  if constexpr (ACT == KMIP_ACT_RELU) return z < 0.f ? 0.f : z;
  return z;
}

// act(z) and act'(z); relu'(0) = 0.
template <typename T, int ACT>
__device__ __forceinline__ void act_both(float z, float& f, float& g) {
  if constexpr (ACT == KMIP_ACT_SILU) {
    const float s = sigmoid<T>(z);
    f = z * s;
    g = fmaf(f, 1.f - s, s);
  } else if constexpr (ACT == KMIP_ACT_GELU) {
    float c, d;
    gauss<T>(z, c, d);
    f = z * c;
    g = fmaf(z, d, c);
  } else if constexpr (ACT == KMIP_ACT_RELU) {
    f = z < 0.f ? 0.f : z;
    g = z > 0.f ? 1.f : 0.f;
  } else {
    f = z;
    g = 1.f;
  }
}

// Two values at a time: sm_100's packed fp32 instructions, each half rounded as
// the single one would be.
__device__ __forceinline__ uint64_t as_u64(float2 v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
  return r;
}
__device__ __forceinline__ float2 as_f2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ float2 splat2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(as_u64(a)), "l"(as_u64(b)));
  return as_f2(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(r)
      : "l"(as_u64(a)), "l"(as_u64(b)), "l"(as_u64(c)));
  return as_f2(r);
}

// Sigmoids of two values, z limited from below to kLeast first (silu(kLeast) is
// -3e-18).  bf16: both quotients out of one reciprocal, of the product of the
// denominators, which that limit keeps under 2^127: three slow-pipe
// instructions for two values instead of four.  A NaN stays in z and so in what
// the sigmoid is multiplied with, but is not let into that product, where the
// other value would meet it.
constexpr float kLeast = -44.f;
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2& z) {
  if constexpr (sizeof(T) == 2) {
    constexpr float kLog2e = 1.4426950408889634f;
    const float2 t = mul2(z, splat2(-kLog2e));  // (fminf drops a NaN)
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(z.x) : "f"(kLeast));
    asm("max.NaN.f32 %0, %0, %1;" : "+f"(z.y) : "f"(kLeast));
    const float2 q = add2(make_float2(ex2_fast(fminf(t.x, -kLog2e * kLeast)),
                                      ex2_fast(fminf(t.y, -kLog2e * kLeast))),
                          splat2(1.f));
    const float r = rcp_fast(q.x * q.y);
    return make_float2(q.y * r, q.x * r);
  } else {
    return make_float2(sigmoid<T>(z.x), sigmoid<T>(z.y));
  }
}

template <typename T, int ACT>
__device__ __forceinline__ float2 act_value2(float2 z) {
  if constexpr (ACT == KMIP_ACT_SILU) {
    const float2 s = sigmoid2<T>(z);
    return mul2(z, s);
  }
  return make_float2(act_value<T, ACT>(z.x), act_value<T, ACT>(z.y));
}

template <typename T, int ACT>
__device__ __forceinline__ void act_both2(float2 z, float2& f, float2& g) {
  if constexpr (ACT == KMIP_ACT_SILU) {
    const float2 s = sigmoid2<T>(z);
    f = mul2(z, s);
    g = fma2(f, fma2(s, splat2(-1.f), splat2(1.f)), s);
  } else {
    act_both<T, ACT>(z.x, f.x, g.x);
    act_both<T, ACT>(z.y, f.y, g.y);
  }
}

// Runs f<ACT>() for the run-time code `act` (one uniform branch).
#define KMIP_ACT_SWITCH(act, ...)                                            \
  switch (act) {                                                             \
    case KMIP_ACT_SILU: { constexpr int ACT = KMIP_ACT_SILU; __VA_ARGS__; break; } \
    case KMIP_ACT_GELU: { constexpr int ACT = KMIP_ACT_GELU; __VA_ARGS__; break; } \
    case KMIP_ACT_RELU: { constexpr int ACT = KMIP_ACT_RELU; __VA_ARGS__; break; } \
    default: { constexpr int ACT = KMIP_ACT_NONE; __VA_ARGS__; }             \
  }

}  // namespace kmip
