// quantise.cu -- rows in e4m3 with a scale for each block of 128 columns, the x of molora_linear_blocks:
//
//   scale8[t,b] = max(max_{i in b} |x[t,i]|, 2^-64) / 448,    out8[t,i] = x[t,i] / scale8[t,b]
//
// Both quotients round as fp32 divisions do: bf16's eight bits over a scale made of another eight often fall halfway between two
// e4m3 values, where the product with a rounded reciprocal, a step of fp32 off, takes the other one (1 in 2000).
// Bound by HBM: bf16 takes 3 bytes an element (8192 x 4096: 17.8 us, 5710 GB/s).  A block is 16 lanes of 8 elements, so a lane's elements are one
// or two 16-byte loads and one 8-byte store, and the largest value takes 4 shuffles.  A warp takes kUnits pieces of two
// blocks in a row, all of whose loads are in flight together.
#include "linear.cuh"

namespace molora {

namespace {

constexpr int kThreadsQ = 256;
constexpr int kBlock = 128;

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// x / s from inv, 1 / s rounded, and minus = -s: the product with inv, corrected by what it leaves of x (Markstein, 1990); for two
// x in one instruction each.  Three operations for a product's one, but with the scale made so too, in place of the compiler's
// division, 8192 x 4096 bf16 takes 17.75 us where it took 18.5 (16384 x 512 6.3, 6.1).  -0 becomes 0.
__device__ __forceinline__ float divide(float x, float inv, float minus) {
  const float q = x * inv;
  return fmaf(fmaf(q, minus, x), inv, q);
}
__device__ __forceinline__ void divide_pair(float& a, float& b, float inv, float minus) {
  asm("{\n\t.reg .b64 x, i, m, q, r;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 i, {%2, %2};\n\tmov.b64 m, {%3, %3};\n\t"
      "mul.rn.f32x2 q, x, i;\n\tfma.rn.f32x2 r, q, m, x;\n\tfma.rn.f32x2 q, r, i, q;\n\tmov.b64 {%0, %1}, q;\n\t}"
      : "+f"(a), "+f"(b)
      : "f"(inv), "f"(minus));
}

// Eight elements of a row: as they are loaded, their largest magnitude (over the 16 lanes of a block), and as floats.
template <typename T>
struct Eight;

template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) { a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1]; }
  __device__ __forceinline__ void load(const float* p, int left) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.f;
    a = make_float4(v[0], v[1], v[2], v[3]), b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ float largest() const {
    float m = max_nan(max_nan(max_nan(fabsf(a.x), fabsf(a.y)), max_nan(fabsf(a.z), fabsf(a.w))),
                      max_nan(max_nan(fabsf(b.x), fabsf(b.y)), max_nan(fabsf(b.z), fabsf(b.w))));
#pragma unroll
    for (int off = 8; off; off >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, off, 16));
    return m;
  }
};

template <>
struct Eight<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int left) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < left ? (uint32_t)__bfloat16_as_ushort(p[i]) : 0u;
    q = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
  __device__ __forceinline__ float largest() const {
    constexpr uint32_t kAbs = 0x7fff7fffu;
    uint32_t m = max_nan_bf16x2(max_nan_bf16x2(q.x & kAbs, q.y & kAbs), max_nan_bf16x2(q.z & kAbs, q.w & kAbs));
#pragma unroll
    for (int off = 8; off; off >>= 1) m = max_nan_bf16x2(m, __shfl_xor_sync(0xffffffffu, m, off, 16));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
  }
};

}  // namespace

// kVec: rows of x on 16-byte and of out8 on 8-byte boundaries.  Warp w takes piece w % pieces of row w / pieces: kUnits times
// 256 columns.
template <typename T, bool kVec, int kUnits>
__global__ void __launch_bounds__(kThreadsQ)
    quantise_blocks_kernel(const T* __restrict__ x, int64_t warps, int32_t d, int32_t pieces, uint8_t* __restrict__ out8,
                           float* __restrict__ scale8) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * (kThreadsQ / 32) + (threadIdx.x >> 5);
  if (w >= warps) return;
  const int64_t row = warps <= UINT32_MAX ? (uint32_t)w / (uint32_t)pieces : w / pieces;
  const int32_t col0 = (int32_t)(w - row * pieces) * (kUnits * 256) + lane * 8, blocks = (d - 1) / kBlock + 1;
  const T* p = x + row * d;
  Eight<T> e[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int32_t col = col0 + k * 256;
    if (kVec && col + 8 <= d)
      e[k].load(p + col);
    else
      e[k].load(p + col, d - col);
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int32_t col = col0 + k * 256;
    const float most = max_nan(e[k].largest(), 0x1p-64f);
    const bool finite = most < __uint_as_float(0x7f800000u);  // (else there is nothing to correct by)
    const float scale = finite ? divide(most, 1.f / 448.f, -448.f) : most, inv = 1.f / scale;
    if (col >= d) continue;  // (columns past 2^31 - 1 there are none: d is below 2^31 - 1023)
    if ((lane & 15) == 0) scale8[row * blocks + col / kBlock] = scale;
    const float minus = finite ? -scale : 0.f;
    float v[8];
    e[k].values(v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) divide_pair(v[i], v[i + 1], inv, minus);
    uint32_t packed[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = {v[4 * i], v[4 * i + 1]}, b = {v[4 * i + 2], v[4 * i + 3]};
      packed[i] = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
                  (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
    }
    uint8_t* o = out8 + row * d + col;
    if (kVec && col + 8 <= d) {
      *reinterpret_cast<uint2*>(o) = make_uint2(packed[0], packed[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (col + i < d) o[i] = (uint8_t)(packed[i / 4] >> (8 * (i & 3)));
    }
  }
}

namespace {

template <typename T>
cudaError_t launch_typed(const T* x, int64_t N, int32_t d, void* out8, float* scale8, cudaStream_t stream) {
  const bool vec = (int64_t)d * sizeof(T) % 16 == 0 && d % 8 == 0 && aligned(x, 16) && aligned(out8, 8);
  auto go = [&](auto kernel, int units) {
    const int32_t pieces = (d - 1) / (units * 256) + 1;
    const int64_t warps = N * pieces, grid = (warps + kThreadsQ / 32 - 1) / (kThreadsQ / 32);
    if (grid > INT32_MAX) return cudaErrorNotSupported;
    return launch_kernel(kernel, dim3((unsigned)grid), dim3(kThreadsQ), 0, stream, 0, x, warps, d, pieces,
                         static_cast<uint8_t*>(out8), scale8);
  };
  // one piece a warp where rows are short or few, so that they spread over the SMs
  if (d <= 512 || N * d <= (int64_t)num_sms() * 32 * 1024)
    return vec ? go(quantise_blocks_kernel<T, true, 1>, 1) : go(quantise_blocks_kernel<T, false, 1>, 1);
  return vec ? go(quantise_blocks_kernel<T, true, 4>, 4) : go(quantise_blocks_kernel<T, false, 4>, 4);
}

}  // namespace

cudaError_t launch_quantise_blocks(const void* x, molora_dtype dtype, int64_t N, int32_t d, void* out8, float* scale8,
                                   cudaStream_t stream) {
  if (dtype == MOLORA_BF16) return launch_typed(static_cast<const __nv_bfloat16*>(x), N, d, out8, scale8, stream);
  return launch_typed(static_cast<const float*>(x), N, d, out8, scale8, stream);
}

}  // namespace molora
