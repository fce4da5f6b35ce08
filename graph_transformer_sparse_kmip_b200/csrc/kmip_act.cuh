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

__device__ __forceinline__ float gauss_cdf(float z) {
  return 0.5f * erfcf(-0.70710678118654752f * z);
}

template <typename T>
__device__ __forceinline__ float gauss_pdf(float z) {
  const float e = -0.5f * z * z;
  return 0.39894228040143268f * (sizeof(T) == 2 ? __expf(e) : expf(e));
}

// act(z).  relu passes a NaN on.
template <typename T, int ACT>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (ACT == KMIP_ACT_SILU) return z * sigmoid<T>(z);
  if constexpr (ACT == KMIP_ACT_GELU) return z * gauss_cdf(z);
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
    const float c = gauss_cdf(z);
    f = z * c;
    g = fmaf(z, gauss_pdf<T>(z), c);
  } else if constexpr (ACT == KMIP_ACT_RELU) {
    f = z < 0.f ? 0.f : z;
    g = z > 0.f ? 1.f : 0.f;
  } else {
    f = z;
    g = 1.f;
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
