// linear.cuh -- what the kernels of the products share: the epilogue's activation, the conversions of its
// element types and its pieces of four outputs, the boxes that operands and outputs move in, tensor maps, and
// how a product splits over clusters.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

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
// normal_tail: Q(z) e^(z^2 / 2), for 0 <= z.
__device__ __forceinline__ float normal_tail(float z) {
  float t;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(0.3f, z, 1.f)));
  float q = 0.0383342616f;
  q = fmaf(q, t, -0.168951929f);
  q = fmaf(q, t, 0.228217259f);
  q = fmaf(q, t, -0.0759995431f);
  q = fmaf(q, t, 0.142185017f);
  q = fmaf(q, t, 0.094832994f);
  q = fmaf(q, t, 0.121882051f);
  q = fmaf(q, t, 0.119493067f);
  q = fmaf(q, t, 6.85289888e-06f);
  return q;
}
__device__ __forceinline__ float gelu_erf(float v) {
  const float z = fminf(fabsf(v), 14.f);
  float e, most;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * (-0.72134752f * z)));
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(most) : "f"(v));
  return fmaf(-z * normal_tail(z), e, most);
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

// act(v) and act'(v) together, from one power each (see activate):
//   SiLU        p = 1 / (1 + 2^(-v log2 e)):  v p,  p + v p (1 - p)
//   GELU        Phi(v) the normal distribution, phi(v) its density:  v Phi(v),  Phi(v) + v phi(v)
//   GELU, tanh  p = 1 / (1 + 2^(-2 u log2 e)):  v p,  p + v p (1 - p) 2 u',  u' = sqrt(2 / pi) (1 + 0.134145 v^2)
// 1 - p is the power times p where p is near 1, which leaves nothing to cancel.  Where 2^z overflows p is 0, and so are
// both; v^2 is kept finite, so that nothing there is 0 times infinity.
__device__ __forceinline__ void act_and_slope(float v, molora_activation act, float& a, float& s) {
  auto exp2_fast = [](float z) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z));
    return e;
  };
  auto sigmoid = [](float e) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
  };
  switch (act) {
    case MOLORA_ACT_RELU:
      a = v > 0.f ? v : (v != v ? v : 0.f);
      s = v > 0.f ? 1.f : (v != v ? v : 0.f);
      return;
    case MOLORA_ACT_SILU: {
      const float e = exp2_fast(-1.4426950408889634f * v), p = sigmoid(e);
      a = v * p;
      s = fmaf(a, e < 1.f ? e * p : 1.f - p, p);
      return;
    }
    case MOLORA_ACT_GELU_TANH: {
      const float e = exp2_fast(v * fmaf(-0.10294324f * v, v, -2.3022082f)), p = sigmoid(e);
      a = v * p;
      s = fmaf(a, (e < 1.f ? e * p : 1.f - p) * fmaf(0.21406859f, fminf(v * v, 1e30f), 1.5957691f), p);
      return;
    }
    case MOLORA_ACT_GELU: {
      a = gelu_erf(v);
      const float z = fminf(fabsf(v), 14.f), e = exp2_fast(z * (-0.72134752f * z)), tail = normal_tail(z) * e;
      s = fmaf(copysignf(z, v), 0.3989422804f * e, v > 0.f ? 1.f - tail : tail);
      if (v != v) s = v;
      return;
    }
    default:
      a = v;
      s = 1.f;
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

// As umma_stage of bf16, with the 16-byte units between the steps of A too.
#define MOLORA_UMMA4_STEPS(group)                                                                                        \
  asm volatile(                                                                                                          \
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t.reg .b32 al, bl;\n\t"                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                                                        \
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %4};\n\t"                                                               \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], da, db, %5, p;\n\t"                                              \
      "setp.eq.b32 p, 0, 0;\n\t"                                                                                         \
      "add.u32 al, %1, %7;\n\tadd.u32 bl, %2, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"                 \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], da, db, %5, p;\n\t"                                              \
      "add.u32 al, al, %7;\n\tadd.u32 bl, bl, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"                 \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], da, db, %5, p;\n\t"                                              \
      "add.u32 al, al, %7;\n\tadd.u32 bl, bl, %8;\n\tmov.b64 da, {al, %3};\n\tmov.b64 db, {bl, %4};\n\t"                 \
      "tcgen05.mma.cta_group::" group ".kind::f16 [%0], da, db, %5, p;\n\t}" ::"r"(d),                                   \
      "r"(a), "r"(b), "r"(a_hi), "r"(b_hi), "r"(idesc), "r"(accumulate), "r"(a_step), "r"(b_step)                        \
      : "memory")

template <bool kPair>
__device__ __forceinline__ void umma_stage_steps(uint32_t d, uint32_t a, uint32_t b, uint32_t a_hi, uint32_t b_hi, uint32_t idesc,
                                                 uint32_t accumulate, uint32_t a_step, uint32_t b_step) {
  if constexpr (kPair)
    MOLORA_UMMA4_STEPS("2");
  else
    MOLORA_UMMA4_STEPS("1");
}
#undef MOLORA_UMMA4_STEPS

constexpr uint32_t kAtom = 64 * 128;  // a box of 64 columns x 64 rows of K, of an operand that lies MN-major
constexpr int kRows = 128;          // rows of a box of x (or of W in the skinny kernels) = TMEM lanes
constexpr uint32_t kRowBytes = 128; // bytes of K per stage
// More bytes in flight take longer to come: one token, 4096 x 4096 bf16 from HBM 9.4 us with 4 stages, 8.8
// with 8, 10.0 with 12 (from L2 7.1, 7.4, 8.2).
constexpr int kMaxStages = 8;
// K blocks of 64 bf16 that many tokens' kernels with 16-bit outputs sum in TMEM before fp32 registers take over.  A tensor core's
// additions cut what they lose, so sums of one sign come out short, the more the longer the chain: measured 1.0e-5 after 64
// blocks, 2.9e-5 after 128, 7.5e-5 after 256, 1.6e-3 (four tenths of bf16's half step, for every output) after 4096, which 2^18
// tokens' dW is.  At 128 taking the chains costs nothing that shows (16000 tokens, 4096 -> 8192 3709 us for both gradients, 3694
// in one chain, 3747 in chains of 64).  Sums that are no longer, those of most calls, keep nothing in registers.
constexpr int kChain = 128;
constexpr uint32_t kTurn = 4096;    // 32 x 32 values of fp32 y
constexpr size_t kMaxSmem = 227 * 1024;
constexpr size_t kSmemSlack = 1024;
constexpr uint32_t kBox = 2048;     // of the epilogue's staging: 32 rows x 64 bytes

template <int N>
__device__ __forceinline__ void apply_act(float (&v)[N], molora_activation act) {
  if (act == MOLORA_ACT_NONE) return;
  if (act == MOLORA_ACT_RELU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOLORA_ACT_RELU);
  } else if (act == MOLORA_ACT_SILU) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOLORA_ACT_SILU);
  } else if (act == MOLORA_ACT_GELU_TANH) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOLORA_ACT_GELU_TANH);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate(v[i], MOLORA_ACT_GELU);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Four consecutive outputs o .. o + 3 of a token as the epilogue reads and writes them: in one access
// where `vec` (rows of 4-element pieces on 16-byte boundaries), else one by one, those past d_out left out.
struct Quad {
  float v[4];
  __device__ __forceinline__ void load(const float* p, int o, int d_out, bool vec) {
    if (vec) {
      const float4 q = *reinterpret_cast<const float4*>(p + o);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = o + i < d_out ? p[o + i] : 0.f;
    }
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int o, int d_out, bool vec) {
    if (vec) {
      const uint2 q = *reinterpret_cast<const uint2*>(p + o);
      v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
      v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = o + i < d_out ? __bfloat162float(p[o + i]) : 0.f;
    }
  }
  __device__ __forceinline__ void store(float* p, int o, int d_out, bool vec) const {
    if (vec) {
      *reinterpret_cast<float4*>(p + o) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (o + i < d_out) p[o + i] = v[i];
    }
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p, int o, int d_out, bool vec) const {
    if (vec) {
      *reinterpret_cast<uint2*>(p + o) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (o + i < d_out) p[o + i] = __float2bfloat16_rn(v[i]);
    }
  }
};

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline uint32_t tmem_columns(uint32_t n) {
  uint32_t c = 32;
  while (c < n) c *= 2;
  return c;
}

// A tensor map of `rows` dense rows of `cols` elements of esize bytes, in boxes of box_rows x box_cols.  False if the
// driver makes none of it.
bool linear_map(CUtensorMap* m, CUtensorMapDataType type, uint32_t esize, const void* base, uint64_t rows, uint64_t cols,
                uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swz);
// The same of three dimensions, the densest first; step: the bytes from one element of the second, and of the third, to
// the next.
bool linear_map_3d(CUtensorMap* m, CUtensorMapDataType type, const void* base, const uint64_t (&size)[3],
                   const uint64_t (&step)[2], const uint32_t (&box)[3], CUtensorMapSwizzle swz);

// How many clusters of 1 to 8 CTAs (one an SM) the current device holds at once: its groups of SMs are not
// multiples of every size (on GB300's 152 SMs: 76 of 2, 36 of 4, 23 of 6, 15 of 8).  Asked for once a
// device; one look at the current device a call, since a small product is over in 4 us.
struct Resident {
  int of[9];
};
Resident resident_clusters();

// How many CTAs share a tile's d_in of nkb blocks: as many as let every tile have its cluster at once,
// two blocks each at least.
inline int split_of(const Resident& r, int64_t tiles, int nkb) {
  for (int C = 8; C > 1; --C)
    if (nkb >= 2 * C && tiles <= r.of[C]) return C;
  return 1;
}

}  // namespace molora
