// linear.cuh -- what the kernels of the base product share: the epilogue's activation and the
// conversions of its element types.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace molora {

__device__ __forceinline__ float to_float(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

__device__ __forceinline__ void store_as(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// act(v) in fp32.  The tanh form of GELU is v * sigmoid(2 u), u = sqrt(2 / pi) (v + 0.044715 v^3).
__device__ __forceinline__ float activate(float v, molora_activation act) {
  switch (act) {
    case MOLORA_ACT_RELU:
      return v > 0.f ? v : (v != v ? v : 0.f);
    case MOLORA_ACT_SILU:
      return v / (1.f + expf(-v));
    case MOLORA_ACT_GELU:
      return 0.5f * v * erfcf(v * -0.70710678118654752f);
    case MOLORA_ACT_GELU_TANH: {
      const float u = 0.79788456080286536f * (v + 0.044715f * v * v * v);
      return v / (1.f + expf(-2.f * u));
    }
    default:
      return v;
  }
}

}  // namespace molora
