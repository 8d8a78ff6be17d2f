// linear.cuh -- what the kernels of the base product share: the epilogue's activation and the
// conversions of its element types.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace molora {

__device__ __forceinline__ float to_float(__nv_fp8_e4m3 v) { return static_cast<float>(v); }

// v / (1 + 2^z) by the hardware's power and reciprocal.  Where 2^z overflows the result is v * 0.
__device__ __forceinline__ float over_one_plus_exp2(float v, float z) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return v * r;
}

// GELU, v (1 + erf(v / sqrt(2))) / 2 = max(v, 0) - z Q(z) with z = |v| and Q(z) = erfc(z / sqrt(2)) / 2, the
// normal distribution's tail.  Q(z) e^(z^2 / 2) falls smoothly from 1/2 and is a polynomial of degree 8 in
// t = 1 / (1 + 0.3 z), fitted here for the least relative error over 0 <= z <= 13.5 (7.9e-8 with the coefficients in
// fp32); past that z Q(z) is below the smallest normal number.  No cancellation: of v < 0 only the second term is left.  17
// instructions an element: 4096 x 2048 -> 6144 in e4m3 takes 47 us with it, 36 with no activation; with erfcf, 115.
__device__ __forceinline__ float gelu_erf(float v) {
  const float z = fminf(fabsf(v), 14.f);
  float t, e, most;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3f, z, 1.f)));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * (-0.72134752f * z)));
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(most) : "f"(v));
  float q = 0.0383342616f;
  q = fmaf(q, t, -0.168951929f);
  q = fmaf(q, t, 0.228217259f);
  q = fmaf(q, t, -0.0759995431f);
  q = fmaf(q, t, 0.142185017f);
  q = fmaf(q, t, 0.094832994f);
  q = fmaf(q, t, 0.121882051f);
  q = fmaf(q, t, 0.119493067f);
  q = fmaf(q, t, 6.85289888e-06f);
  return fmaf(-z * q, e, most);
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
