// rmsnorm.cu -- root-mean-square norm of each row, with the residual's addition before it and an
// optional output in 8 bits:
//
//   s = x + residual                      (fp32; sum_out = s rounded to x's type)
//   n = s * rsqrt(mean(s^2) + eps) * g    (fp32; out = n rounded to x's type)
//   scale8 = max(max |n|, 2^-64) / 448,   out8 = e4m3(n / scale8)
//
// A row is read once: s stays in registers between the reduction and the outputs.  The norm uses
// the unrounded s, so rounding sum_out does not reach the other outputs.
#include <cuda_fp8.h>

#include "common.cuh"
#include "kernels.h"

namespace molora {

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kLowestAmax = 5.421010862427522e-20f;  // 2^-64

// One chunk of a row: 16 bytes of bf16 or fp32, or a single element where rows are not 16-byte
// aligned.
template <typename T, bool kVec>
struct Chunk;
template <>
struct Chunk<__nv_bfloat16, true> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Chunk<float, true> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void load(const float* p, float (&v)[4]) {
    const float4 u = *reinterpret_cast<const float4*>(p);
    v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, false> {
  static constexpr int n = 1;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&v)[1]) { v[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[1]) { *p = __float2bfloat16_rn(v[0]); }
};
template <>
struct Chunk<float, false> {
  static constexpr int n = 1;
  static __device__ __forceinline__ void load(const float* p, float (&v)[1]) { v[0] = *p; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[1]) { *p = v[0]; }
};

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[8], float f) {
  *reinterpret_cast<uint2*>(p) = make_uint2(e4m3x2(v[0] * f, v[1] * f) | (e4m3x2(v[2] * f, v[3] * f) << 16),
                                            e4m3x2(v[4] * f, v[5] * f) | (e4m3x2(v[6] * f, v[7] * f) << 16));
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[4], float f) {
  *reinterpret_cast<uint32_t*>(p) = e4m3x2(v[0] * f, v[1] * f) | (e4m3x2(v[2] * f, v[3] * f) << 16);
}
__device__ __forceinline__ void store8(uint8_t* p, const float (&v)[1], float f) {
  *p = (uint8_t)__nv_cvt_float_to_fp8(v[0] * f, __NV_SATFINITE, __NV_E4M3);
}

template <typename T>
struct NormArgs {
  const T* x;
  const T* res;
  T* sum_out;
  const T* g;
  T* out;
  uint8_t* out8;
  float* scale8;
  int64_t N;
  int32_t d;
  float eps;
};

// Sum and maximum over the `warps` warps of a team; red holds 2 floats per warp of the CTA, the
// team's first at red[2 * warp0].  Called by every thread of the CTA.
__device__ __forceinline__ void team_reduce(float& sum, float& top, int warps, int warp0, float* red) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[2 * warp] = sum, red[2 * warp + 1] = top;
  __syncthreads();
  sum = 0.f, top = 0.f;
  for (int i = 0; i < warps; ++i) sum += red[2 * (warp0 + i)], top = fmaxf(top, red[2 * (warp0 + i) + 1]);
  __syncthreads();
}

// The 8-bit scale of a row whose largest |s * g| is `top`.  A NaN stays one.
__device__ __forceinline__ float row_scale(float top, float inv) {
  const float amax = top * inv;
  return (amax < kLowestAmax ? kLowestAmax : amax) / kE4m3Max;
}

}  // namespace

// `team` threads (32 .. the CTA's) a row, up to NC chunks of it held by each thread.  kRagged: d is
// not a multiple of the chunk, so rows start anywhere in the arrays' 16-byte grid; a row's chunks
// are those of the grid it touches, its first and last ones handled element by element.
template <typename T, bool kVec, int NC, bool kRagged>
__global__ void __launch_bounds__(1024) rmsnorm_kernel(const NormArgs<T> a, int team) {
  using C = Chunk<T, kVec>;
  __shared__ float red[64];
  const int in_team = threadIdx.x & (team - 1), which = threadIdx.x / team, teams = blockDim.x / team;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * teams;
  for (int64_t t0 = (int64_t)blockIdx.x * teams; t0 < a.N; t0 += step) {
    const int64_t t = t0 + which;
    const bool live = t < a.N;
    const int shift = kRagged ? (int)((t * a.d) & (C::n - 1)) : 0;
    const int chunks = live ? (a.d + shift + C::n - 1) / C::n : 0;
    const int64_t base = t * a.d - shift;  // the first chunk's place in the arrays
    auto whole = [&](int c) { return !kRagged || (c * C::n >= shift && (c + 1) * C::n <= a.d + shift); };
    auto inside = [&](int c, int j) { return c * C::n + j >= shift && c * C::n + j < a.d + shift; };
    auto load = [&](const T* p, int c, float (&v)[C::n]) {
      if (whole(c)) {
        C::load(p + base + (int64_t)c * C::n, v);
      } else {
#pragma unroll
        for (int j = 0; j < C::n; ++j) v[j] = inside(c, j) ? to_float(p[base + (int64_t)c * C::n + j]) : 0.f;
      }
    };
    auto store = [&](T* p, int c, const float (&v)[C::n]) {
      if (whole(c)) {
        C::store(p + base + (int64_t)c * C::n, v);
      } else {
#pragma unroll
        for (int j = 0; j < C::n; ++j) {
          const float one[1] = {v[j]};
          if (inside(c, j)) Chunk<T, false>::store(p + base + (int64_t)c * C::n + j, one);
        }
      }
    };
    float s[NC][C::n];
    float sum = 0.f, top = 0.f;
    // every load of the row is in flight before the first is used
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c < chunks) load(a.x, c, s[i]);
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = in_team + i * team;
        if (c < chunks) {
          float r[C::n];
          load(a.res, c, r);
#pragma unroll
          for (int j = 0; j < C::n; ++j) s[i][j] += r[j];
        }
      }
      if (a.sum_out) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (in_team + i * team < chunks) store(a.sum_out, in_team + i * team, s[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c < chunks) {
        float g[C::n];
        if (kRagged) {
#pragma unroll
          for (int j = 0; j < C::n; ++j) g[j] = inside(c, j) ? to_float(a.g[c * C::n + j - shift]) : 0.f;
        } else {
          C::load(a.g + (int64_t)c * C::n, g);
        }
#pragma unroll
        for (int j = 0; j < C::n; ++j) {
          sum = fmaf(s[i][j], s[i][j], sum);
          s[i][j] *= g[j];
          top = fmaxf(top, fabsf(s[i][j]));
        }
      }
    }
    team_reduce(sum, top, team / 32, which * (team / 32), red);
    const float inv = 1.f / sqrtf(sum / (float)a.d + a.eps);
    const float scale = row_scale(top, inv), f8 = 1.f / scale;
    if (live && a.out8 && in_team == 0) a.scale8[t] = scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c < chunks) {
#pragma unroll
        for (int j = 0; j < C::n; ++j) s[i][j] *= inv;
        if (a.out) store(a.out, c, s[i]);
        if (a.out8) {
          if (whole(c)) {
            store8(a.out8 + base + (int64_t)c * C::n, s[i], f8);
          } else {
#pragma unroll
            for (int j = 0; j < C::n; ++j) {
              const float one[1] = {s[i][j]};
              if (inside(c, j)) store8(a.out8 + base + (int64_t)c * C::n + j, one, f8);
            }
          }
        }
      }
    }
  }
}

// Rows too long for one CTA's registers: x and residual are read again (from L2) for the outputs,
// element by element, so each output may only be the input it replaces element for element.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormArgs<T> a) {
  __shared__ float red[64];
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < a.N; t += gridDim.x) {
    const int64_t base = t * a.d;
    float sum = 0.f, top = 0.f;
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float s = to_float(a.x[base + c]);
      if (a.res) s += to_float(a.res[base + c]);
      sum = fmaf(s, s, sum);
      top = fmaxf(top, fabsf(s * to_float(a.g[c])));
    }
    team_reduce(sum, top, blockDim.x / 32, 0, red);
    const float inv = 1.f / sqrtf(sum / (float)a.d + a.eps);
    const float scale = row_scale(top, inv), f8 = 1.f / scale;
    if (a.out8 && threadIdx.x == 0) a.scale8[t] = scale;
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float s = to_float(a.x[base + c]);
      if (a.res) s += to_float(a.res[base + c]);
      const float n[1] = {s * to_float(a.g[c]) * inv}, sv[1] = {s};
      if (a.sum_out) Chunk<T, false>::store(a.sum_out + base + c, sv);
      if (a.out) Chunk<T, false>::store(a.out + base + c, n);
      if (a.out8) store8(a.out8 + base + c, n, f8);
    }
  }
}

namespace {

constexpr int kFew = 2;

template <typename T, bool kVec, bool kRagged>
cudaError_t launch_norm(const NormArgs<T>& a, cudaStream_t stream) {
  const int64_t chunks = (a.d + Chunk<T, kVec>::n - 1) / Chunk<T, kVec>::n + (kRagged ? 1 : 0);
  // few chunks a thread where there are few rows (one row's latency), up to kFew where there are many
  int team = 32;
  while (team < 1024 && chunks > (int64_t)team * kFew) team *= 2;
  while (team < 1024 && chunks > team && a.N * team * 2 <= (int64_t)num_sms() * 1024) team *= 2;
  const int per = (int)((chunks + team - 1) / team);
  const int threads = team < 256 ? 256 : team;
  const int64_t groups = (a.N + threads / team - 1) / (threads / team);
  const int64_t most = (int64_t)num_sms() * (2048 / threads);
  const dim3 grid((unsigned)(groups < most ? groups : most)), block(threads);
  if (per <= 1) return launch_kernel(rmsnorm_kernel<T, kVec, 1, kRagged>, grid, block, 0, stream, 0, a, team);
  if (per <= 2) return launch_kernel(rmsnorm_kernel<T, kVec, 2, kRagged>, grid, block, 0, stream, 0, a, team);
  if (per <= 4) return launch_kernel(rmsnorm_kernel<T, kVec, 4, kRagged>, grid, block, 0, stream, 0, a, team);
  if (Chunk<T, kVec>::n <= 4 && per <= 8)
    return launch_kernel(rmsnorm_kernel<T, kVec, Chunk<T, kVec>::n <= 4 ? 8 : 4, kRagged>, grid, block, 0, stream, 0, a, team);
  const dim3 rows((unsigned)(a.N < 2 * num_sms() ? a.N : 2 * num_sms()));
  return launch_kernel(rmsnorm_long_kernel<T>, rows, dim3(1024), 0, stream, 0, a);
}

template <typename T>
cudaError_t launch_norm_typed(const void* x, int64_t N, int32_t d, const void* residual, void* sum_out,
                              const void* weight, float eps, void* out, void* out8, float* scale8,
                              cudaStream_t stream) {
  const NormArgs<T> a = {static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<T*>(sum_out),
                         static_cast<const T*>(weight), static_cast<T*>(out), static_cast<uint8_t*>(out8), scale8, N, d,
                         eps};
  const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(residual) |
                         reinterpret_cast<uintptr_t>(sum_out) | reinterpret_cast<uintptr_t>(weight) |
                         reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(out8);
  if (bits & 15u) return launch_norm<T, false, false>(a, stream);
  return d % Chunk<T, true>::n ? launch_norm<T, true, true>(a, stream) : launch_norm<T, true, false>(a, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, molora_dtype dtype, int64_t N, int32_t d, const void* residual, void* sum_out,
                           const void* weight, float eps, void* out, void* out8, float* scale8, cudaStream_t stream) {
  if (dtype == MOLORA_BF16)
    return launch_norm_typed<__nv_bfloat16>(x, N, d, residual, sum_out, weight, eps, out, out8, scale8, stream);
  return launch_norm_typed<float>(x, N, d, residual, sum_out, weight, eps, out, out8, scale8, stream);
}

}  // namespace molora
