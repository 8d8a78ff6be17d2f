// quantise.cu -- rows in e4m3 with a scale for each block of 128 columns, the x of molora_linear_blocks:
//
//   scale8[t,b] = max(max_{i in b} |x[t,i]|, 2^-64) / 448,    out8[t,i] = x[t,i] * (1 / scale8[t,b])
//
// Bound by HBM: bf16 takes 3 bytes an element.  A block is 16 lanes of 8 elements, so a lane's elements are one
// or two 16-byte loads and one 8-byte store, and the largest value takes 4 shuffles.  kUnits blocks' loads are in
// flight a lane, which is what the bandwidth takes.
#include "linear.cuh"

namespace molora {

namespace {

constexpr int kThreadsQ = 256;
constexpr int kBlock = 128;

struct Eight {
  float v[8];
};

__device__ __forceinline__ void load_eight(const float* p, Eight& e) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  e.v[0] = a.x, e.v[1] = a.y, e.v[2] = a.z, e.v[3] = a.w, e.v[4] = b.x, e.v[5] = b.y, e.v[6] = b.z, e.v[7] = b.w;
}
__device__ __forceinline__ void load_eight(const __nv_bfloat16* p, Eight& e) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) e.v[2 * i] = __uint_as_float(w[i] << 16), e.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
}

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace

// kVec: rows of x on 16-byte and of out8 on 8-byte boundaries.  Unit u: row u / blocks, block u % blocks.
template <typename T, bool kVec, int kUnits>
__global__ void __launch_bounds__(kThreadsQ)
    quantise_blocks_kernel(const T* __restrict__ x, int64_t units, int32_t d, int32_t blocks, uint8_t* __restrict__ out8,
                           float* __restrict__ scale8) {
  pdl_wait();
  pdl_launch_dependents();
  const int lane16 = threadIdx.x & 15;
  constexpr int kGroups = kThreadsQ / 16;
  const int64_t first = (int64_t)blockIdx.x * (kGroups * kUnits) + (threadIdx.x >> 4);
  Eight e[kUnits];
  int64_t row[kUnits];
  int col[kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int64_t u = first + k * kGroups;
    row[k] = u / blocks;
    col[k] = (int)(u - row[k] * blocks) * kBlock + lane16 * 8;
    const int left = u < units ? d - col[k] : 0;
    const T* p = x + row[k] * d + col[k];
    if (kVec && left >= 8) {
      load_eight(p, e[k]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[k].v[i] = i < left ? to_float(p[i]) : 0.f;
    }
  }
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int64_t u = first + k * kGroups;
    float most = 0x1p-64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max_nan(most, fabsf(e[k].v[i]));
#pragma unroll
    for (int off = 8; off; off >>= 1) most = max_nan(most, __shfl_xor_sync(0xffffffffu, most, off, 16));
    const float scale = most / 448.f, inv = 1.f / scale;
    const int left = u < units ? d - col[k] : 0;
    if (u < units && lane16 == 0) scale8[u] = scale;
    uint32_t packed[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float2 a = {e[k].v[4 * i] * inv, e[k].v[4 * i + 1] * inv}, b = {e[k].v[4 * i + 2] * inv, e[k].v[4 * i + 3] * inv};
      packed[i] = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
                  (uint32_t)__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3) << 16;
    }
    uint8_t* o = out8 + row[k] * d + col[k];
    if (kVec && left >= 8) {
      *reinterpret_cast<uint2*>(o) = make_uint2(packed[0], packed[1]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) o[i] = (uint8_t)(packed[i / 4] >> (8 * (i & 3)));
    }
  }
}

namespace {

template <typename T>
cudaError_t launch_typed(const T* x, int64_t N, int32_t d, void* out8, float* scale8, cudaStream_t stream) {
  constexpr int kUnits = sizeof(T) == 2 ? 4 : 2;
  const int32_t blocks = (int32_t)(((int64_t)d + kBlock - 1) / kBlock);
  const int64_t units = N * blocks;
  const bool vec = (int64_t)d * sizeof(T) % 16 == 0 && d % 8 == 0 && aligned(x, 16) && aligned(out8, 8);
  auto go = [&](auto kernel, int each) {
    const int64_t grid = (units + each - 1) / each;
    if (grid > INT32_MAX) return cudaErrorNotSupported;
    return launch_kernel(kernel, dim3((unsigned)grid), dim3(kThreadsQ), 0, stream, 0, x, units, d, blocks,
                         static_cast<uint8_t*>(out8), scale8);
  };
  constexpr int kGroups = kThreadsQ / 16;
  // few blocks: one a lane group, so that they spread over the SMs
  if (units <= (int64_t)num_sms() * kGroups * kUnits)
    return vec ? go(quantise_blocks_kernel<T, true, 1>, kGroups) : go(quantise_blocks_kernel<T, false, 1>, kGroups);
  return vec ? go(quantise_blocks_kernel<T, true, kUnits>, kGroups * kUnits)
             : go(quantise_blocks_kernel<T, false, kUnits>, kGroups * kUnits);
}

}  // namespace

cudaError_t launch_quantise_blocks(const void* x, molora_dtype dtype, int64_t N, int32_t d, void* out8, float* scale8,
                                   cudaStream_t stream) {
  if (dtype == MOLORA_BF16) return launch_typed(static_cast<const __nv_bfloat16*>(x), N, d, out8, scale8, stream);
  return launch_typed(static_cast<const float*>(x), N, d, out8, scale8, stream);
}

}  // namespace molora
