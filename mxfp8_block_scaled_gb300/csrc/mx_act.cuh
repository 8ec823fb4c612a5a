// Activations of the GEMM epilogue and their derivatives, in FP32 (mx_act of
// include/mxfp8.h), two values at a time for the packed FP32 instructions. GELU
// is the tanh form: 0.5 z (1 + tanh(a (z + b z^3))), a = sqrt(2/pi), b =
// 0.044715, written as z * q with q the logistic function of u = 2 a (z + b
// z^3) (the same expression: (1 + tanh(t))/2 = logistic(2t)), so it shares
// SiLU's form z * logistic(u), u = z, and keeps its relative accuracy where the
// tanh form cancels. q = 1 / (1 + 2^(-u log2 e)) takes two special-function
// instructions, whose rate (a quarter of the others') bounds these functions;
// their error and the exponent's rounding, |u| 2^-23, stay below 2^-16 of the
// result for |u| < 88, far below the BF16 rounding that follows. Results below
// 2^-126 are flushed to zero.
#pragma once

#include <cuda_runtime.h>

#include "../../include/mxfp8.h"

namespace mx {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kGeluU1 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluU3 = 0.07135481627159915f;  // the same times 0.044715

// 1 / (1 + 2^v) of both
__device__ __forceinline__ float2 logistic_of_minus(float2 v) {
  float2 e, q;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(v.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(e.y));
  return q;
}

__device__ __forceinline__ float2 act_pair(float v) { return make_float2(v, v); }

template <int kAct>
__device__ __forceinline__ float2 act_value(float2 z) {
  if constexpr (kAct == MX_ACT_RELU) return make_float2(z.x <= 0.0f ? 0.0f : z.x, z.y <= 0.0f ? 0.0f : z.y);
  if constexpr (kAct == MX_ACT_GELU) {
    const float2 t = __ffma2_rn(__fmul2_rn(z, z), act_pair(-kGeluU3 * kLog2e), act_pair(-kGeluU1 * kLog2e));
    return __fmul2_rn(z, logistic_of_minus(__fmul2_rn(z, t)));
  }
  if constexpr (kAct == MX_ACT_SILU) return __fmul2_rn(z, logistic_of_minus(__fmul2_rn(z, act_pair(-kLog2e))));
  return z;
}

// d act / dz: q + z u' q (1 - q). z u' overflows where q has long been 0 or 1 and
// the product is zero (GELU from |z| = 1.2e13 on; an infinite z), so it is held
// within kSlopeMax: both functions have q (1 - q) = 0 in FP32 well below it (from
// |u| = 88.8 on: |z u'| = 235 for GELU, 89 for SiLU). A NaN comes through by q.
constexpr float kSlopeMax = 1.0e4f;
__device__ __forceinline__ float2 slope_bounded(float2 v) {
  return make_float2(fminf(fmaxf(v.x, -kSlopeMax), kSlopeMax), fminf(fmaxf(v.y, -kSlopeMax), kSlopeMax));
}

template <int kAct>
__device__ __forceinline__ float2 act_slope(float2 z) {
  if constexpr (kAct == MX_ACT_RELU) return make_float2(z.x <= 0.0f ? 0.0f : 1.0f, z.y <= 0.0f ? 0.0f : 1.0f);
  if constexpr (kAct == MX_ACT_GELU || kAct == MX_ACT_SILU) {
    float2 q, zu;  // q, z u'
    if constexpr (kAct == MX_ACT_GELU) {
      const float2 zz = __fmul2_rn(z, z);
      q = logistic_of_minus(__fmul2_rn(z, __ffma2_rn(zz, act_pair(-kGeluU3 * kLog2e), act_pair(-kGeluU1 * kLog2e))));
      zu = __fmul2_rn(z, __ffma2_rn(zz, act_pair(3.0f * kGeluU3), act_pair(kGeluU1)));
    } else {
      q = logistic_of_minus(__fmul2_rn(z, act_pair(-kLog2e)));
      zu = z;
    }
    const float2 rest = __fmul2_rn(q, __ffma2_rn(q, act_pair(-1.0f), act_pair(1.0f)));
    return __ffma2_rn(slope_bounded(zu), rest, q);
  }
  return make_float2(1.0f, 1.0f);
}

// v within kSlopeMax, in one instruction (|v| against it, v's sign).
__device__ __forceinline__ float slope_held(float v) {
  float r;
  asm("min.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(kSlopeMax));
  return r;
}

// act and d act / dz from one logistic function.
template <int kAct>
__device__ __forceinline__ void act_both(float2 z, float2& value, float2& slope) {
  if constexpr (kAct == MX_ACT_GELU || kAct == MX_ACT_SILU) {
    float2 q, zu;
    if constexpr (kAct == MX_ACT_GELU) {
      const float2 zz = __fmul2_rn(z, z);
      q = logistic_of_minus(__fmul2_rn(z, __ffma2_rn(zz, act_pair(-kGeluU3 * kLog2e), act_pair(-kGeluU1 * kLog2e))));
      zu = __fmul2_rn(z, __ffma2_rn(zz, act_pair(3.0f * kGeluU3), act_pair(kGeluU1)));
    } else {
      q = logistic_of_minus(__fmul2_rn(z, act_pair(-kLog2e)));
      zu = z;
    }
    const float2 rest = __fmul2_rn(q, __ffma2_rn(q, act_pair(-1.0f), act_pair(1.0f)));
    slope = __ffma2_rn(make_float2(slope_held(zu.x), slope_held(zu.y)), rest, q);
    value = __fmul2_rn(z, q);
  } else {
    slope = act_slope<kAct>(z);
    value = act_value<kAct>(z);
  }
}

}  // namespace mx
