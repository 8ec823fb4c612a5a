// Activations of the GEMM epilogue and their derivatives, in FP32 (mx_act of
// include/mxfp8.h). GELU is the tanh form: 0.5 z (1 + tanh(a (z + b z^3))), a =
// sqrt(2/pi), b = 0.044715, written as z * q with q the logistic function of
// u = 2 a (z + b z^3) (the same expression: (1 + tanh(t))/2 = logistic(2t)), so
// it shares SiLU's form z * logistic(u), u = z, and keeps its relative accuracy
// where the tanh form cancels. The fast exponential and quotient are off by a
// few 2^-22, far below the BF16 rounding that follows.
#pragma once

#include <cuda_runtime.h>

#include "../../include/mxfp8.h"

namespace mx {

constexpr float kGeluU1 = 1.5957691216057308f;   // 2 sqrt(2/pi)
constexpr float kGeluU3 = 0.07135481627159915f;  // the same times 0.044715

template <int kAct>
__device__ __forceinline__ float act_value(float z) {
  if constexpr (kAct == MX_ACT_RELU) return z <= 0.0f ? 0.0f : z;
  if constexpr (kAct == MX_ACT_GELU) return __fdividef(z, 1.0f + __expf(-z * fmaf(kGeluU3, z * z, kGeluU1)));
  if constexpr (kAct == MX_ACT_SILU) return __fdividef(z, 1.0f + __expf(-z));
  return z;
}

template <int kAct>
__device__ __forceinline__ float act_slope(float z) {
  if constexpr (kAct == MX_ACT_RELU) return z <= 0.0f ? 0.0f : 1.0f;
  if constexpr (kAct == MX_ACT_GELU) {
    const float zz = z * z;
    const float q = __fdividef(1.0f, 1.0f + __expf(-z * fmaf(kGeluU3, zz, kGeluU1)));
    return fmaf(z * fmaf(3.0f * kGeluU3, zz, kGeluU1), q * (1.0f - q), q);
  }
  if constexpr (kAct == MX_ACT_SILU) {
    const float q = __fdividef(1.0f, 1.0f + __expf(-z));
    return fmaf(z, q * (1.0f - q), q);
  }
  return 1.0f;
}

}  // namespace mx
