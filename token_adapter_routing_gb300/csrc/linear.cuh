// linear.cuh -- what the kernels of the base product share: the epilogue's activation and the
// conversions of its element types.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace molora {

__device__ __forceinline__ float to_float(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

// erf's GELU, 32 of which in a row would not fit the registers inline.
static __device__ __noinline__ float gelu_erf(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// v / (1 + exp(-z)).  exp(-z) overflows below z = -88: the quotient is then 0, as for 2^-127.
__device__ __forceinline__ float sigmoid_times(float v, float z) {
  return __fdividef(v, 1.f + __expf(-z));
}

// act(v) in fp32 with the hardware's exponential and reciprocal: a few instructions an element, so
// that the epilogue stays under the MMAs of the next tile.  The tanh form of GELU is v * sigmoid(2 u),
// u = sqrt(2 / pi) (v + 0.044715 v^3).  Their
// relative errors (about 2^-22, plus 2^-24 per unit of the exponent's argument) are below one rounding
// of the sum the value comes from, and 2^13 times below one of a bf16 y.  At large |v| the quotient
// underflows to -0 or tends to v, as the exact forms do.
__device__ __forceinline__ float activate(float v, molora_activation act) {
  switch (act) {
    case MOLORA_ACT_RELU:
      return v > 0.f ? v : (v != v ? v : 0.f);
    case MOLORA_ACT_SILU:
      return sigmoid_times(v, v);
    case MOLORA_ACT_GELU:
      return gelu_erf(v);
    case MOLORA_ACT_GELU_TANH:
      return sigmoid_times(v, 1.5957691216057308f * v * fmaf(0.044715f * v, v, 1.f));
    default:
      return v;
  }
}

}  // namespace molora
