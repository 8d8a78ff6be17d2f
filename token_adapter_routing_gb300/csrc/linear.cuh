// linear.cuh -- what the kernels of the base product share: the epilogue's activation and the
// conversions of its element types.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace molora {

__device__ __forceinline__ float to_float(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

// erf's GELU, 32 of which in a row would not fit the registers inline.
static __device__ __noinline__ float gelu_erf(float v) { return 0.5f * v * erfcf(v * -0.70710678118654752f); }

// v / (1 + 2^z) by the hardware's power and reciprocal.  Where 2^z overflows the result is v * 0.
__device__ __forceinline__ float over_one_plus_exp2(float v, float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return v * r;
}

// act(v) in fp32 with a few instructions an element, so that the epilogue stays under the MMAs of the
// next tile: SiLU is v / (1 + 2^(-v log2 e)), the tanh form of GELU v / (1 + 2^(-2 u log2 e)) with
// u = sqrt(2 / pi) (v + 0.044715 v^3).  The approximations' relative errors (about 2^-22, and 2^-24 per
// unit of the exponent) are below the rounding of the sum that v is, and 2^13 times below one of bf16.
__device__ __forceinline__ float activate(float v, molora_activation act) {
  switch (act) {
    case MOLORA_ACT_RELU:
      return v > 0.f ? v : (v != v ? v : 0.f);
    case MOLORA_ACT_SILU:
      return over_one_plus_exp2(v, -1.4426950408889634f * v);
    case MOLORA_ACT_GELU:
      return gelu_erf(v);
    case MOLORA_ACT_GELU_TANH:
      return over_one_plus_exp2(v, v * fmaf(-0.10294324f * v, v, -2.3022082f));
    default:
      return v;
  }
}

// The MMAs of one stage: 4 steps over K, `a` and `b` the low words of the first step's descriptors (the
// address is all that changes), a_hi and b_hi the high words, b_step 16-byte units between B's steps.
// One asm block: the issuing thread does a handful of dependent integer operations a stage, which is
// what bounds it.  With descriptors built field by field for each MMA a stage took 690 cycles whatever
// the tile's width; a 256 x 256 tile's MMAs take 512.
#define MOLORA_UMMA4(GROUP, KIND)                                                                              \
  asm volatile(                                                                                                \
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t.reg .b32 al, bl;\n\t"                                       \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                              \
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"                                                     \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %5, p;\n\t"                               \
      "setp.eq.b32 p, 0, 0;\n\t"                                                                               \
      "add.u32 al, %1, 2;\n\tadd.u32 bl, %2, %7;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"          \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %5, p;\n\t"                               \
      "add.u32 al, %1, 4;\n\tadd.u32 bl, bl, %7;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"          \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %5, p;\n\t"                               \
      "add.u32 al, %1, 6;\n\tadd.u32 bl, bl, %7;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"          \
      "tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], da, db, %5, p;\n\t}" ::"r"(d),                    \
      "r"(a), "r"(b), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(b_step)                            \
      : "memory")

template <bool kPair, bool kFp8>
__device__ __forceinline__ void umma_stage(uint32_t d, uint32_t a, uint32_t b, uint32_t a_hi, uint32_t b_hi,
                                           uint32_t idesc, uint32_t accumulate, uint32_t b_step = 2) {
  if constexpr (kPair && kFp8)
    MOLORA_UMMA4("2", "f8f6f4");
  else if constexpr (kPair)
    MOLORA_UMMA4("2", "f16");
  else if constexpr (kFp8)
    MOLORA_UMMA4("1", "f8f6f4");
  else
    MOLORA_UMMA4("1", "f16");
}
#undef MOLORA_UMMA4

}  // namespace molora
