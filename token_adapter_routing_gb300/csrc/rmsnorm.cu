// rmsnorm.cu -- root-mean-square norm of each row, with the residual's addition before it and an
// optional output in 8 bits:
//
//   s = x + residual                      (fp32; sum_out = s rounded to x's type)
//   n = s * rsqrt(mean(s^2) + eps) * g    (fp32; out = n rounded to x's type)
//   scale8 = max(max |n|, 2^-64) / 448,   out8 = e4m3(n * (1 / scale8))
//
// A product with the rounded reciprocal, not a quotient: the two differ by 2^-23, so an element that close to a border
// of e4m3, whose own steps are 2^-3, may go to its other side.  A division takes 8192 x 4096 bf16 from 49.0 to 57.5 us
// (with e4m3 alone out from 26.1 to 39.3); a product with one correction, 26.1 to 28.0.
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
    unpack(*reinterpret_cast<const uint4*>(p), v);
  }
  static __device__ __forceinline__ void unpack(const uint4 u, float (&v)[8]) {
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
    unpack(*reinterpret_cast<const uint4*>(p), v);
  }
  static __device__ __forceinline__ void unpack(const uint4 u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
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

// The larger one, or NaN if either is: a row with a NaN has no largest value to scale by.
__device__ __forceinline__ float max_nan(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
  return m;
}

// Sum and maximum over the `warps` warps of a team; red holds 2 floats per warp of the CTA, the
// team's first at red[2 * warp0].  Called by every thread of the CTA; two calls in a row take different
// arrays (a thread may still read one while others write the next).
__device__ __forceinline__ void team_reduce(float& sum, float& top, int warps, int warp0, float* red) {
#pragma unroll
  for (int off = 16; off; off >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, off);
    top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
  }
  if (warps == 1) return;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) red[2 * warp] = sum, red[2 * warp + 1] = top;
  __syncthreads();
  sum = 0.f, top = 0.f;
  for (int i = 0; i < warps; ++i) sum += red[2 * (warp0 + i)], top = max_nan(top, red[2 * (warp0 + i) + 1]);
}

// The 8-bit scale of a row whose largest |s * g| is `top`.  A NaN stays one.
__device__ __forceinline__ float row_scale(float top, float inv) {
  const float amax = top * inv;
  return (amax < kLowestAmax ? kLowestAmax : amax) / kE4m3Max;
}

}  // namespace

// `team` threads (32 .. the CTA's) a row, up to NC chunks of it held by each thread.  kAhead: the next row's
// chunks are on their way while a row is reduced and written (launch_norm says where).  kRagged: d is
// not a multiple of the chunk, so
// rows start anywhere in the arrays' 16-byte grid; a row's chunks are those of the grid it touches, its
// first and last ones handled element by element.
template <typename T, bool kVec, int NC, bool kRagged, bool kAhead>
__global__ void __launch_bounds__(kAhead ? 256 : 1024) rmsnorm_kernel(const NormArgs<T> a, int team) {
  using C = Chunk<T, kVec>;
  __shared__ float red[2][64];
  int turn = 0;
  const int in_team = threadIdx.x & (team - 1), which = threadIdx.x / team, teams = blockDim.x / team;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t step = (int64_t)gridDim.x * teams;
  int shift, chunks;
  int64_t base;  // the first chunk's place in the arrays
  auto place = [&](int64_t t) {
    shift = kRagged ? (int)((t * a.d) & (C::n - 1)) : 0;
    chunks = t < a.N ? (a.d + shift + C::n - 1) / C::n : 0;
    base = t * a.d - shift;
  };
  auto whole = [&](int c) { return C::n == 1 || !kRagged || (c * C::n >= shift && (c + 1) * C::n <= a.d + shift); };
  auto inside = [&](int c, int j) { return c * C::n + j >= shift && c * C::n + j < a.d + shift; };
  uint4 rx[kAhead ? NC : 1], rr[kAhead ? NC : 1];
  auto fetch = [&]() {  // (kAhead: every chunk is whole)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c < chunks) {
        rx[i] = *reinterpret_cast<const uint4*>(a.x + base + (int64_t)c * C::n);
        if (a.res) rr[i] = *reinterpret_cast<const uint4*>(a.res + base + (int64_t)c * C::n);
      }
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
  int64_t t0 = (int64_t)blockIdx.x * teams;
  place(t0 + which);
  if constexpr (kAhead) fetch();
  for (; t0 < a.N; t0 += step) {
    const int64_t t = t0 + which;
    float s[NC][C::n];
    float sum = 0.f, top = 0.f;
    // x's chunks first, then the residual's: all of x is in flight before any of it is used
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c >= chunks) continue;
      if (whole(c)) {
        if constexpr (kAhead)
          C::unpack(rx[i], s[i]);
        else
          C::load(a.x + base + (int64_t)c * C::n, s[i]);
      } else {
#pragma unroll
        for (int j = 0; j < C::n; ++j) s[i][j] = inside(c, j) ? to_float(a.x[base + (int64_t)c * C::n + j]) : 0.f;
      }
    }
    if (a.res) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = in_team + i * team;
        if (c >= chunks) continue;
        float r[C::n];
        if (whole(c)) {
          if constexpr (kAhead)
            C::unpack(rr[i], r);
          else
            C::load(a.res + base + (int64_t)c * C::n, r);
        } else {
#pragma unroll
          for (int j = 0; j < C::n; ++j) r[j] = inside(c, j) ? to_float(a.res[base + (int64_t)c * C::n + j]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < C::n; ++j) s[i][j] += r[j];
      }
    }
    if constexpr (kAhead) {
      place(t + step);
      fetch();
      place(t);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c >= chunks) continue;
      if (a.sum_out) store(a.sum_out, c, s[i]);
      float g[C::n];
      if (kRagged) {
#pragma unroll
        for (int j = 0; j < C::n; ++j) g[j] = inside(c, j) ? to_float(a.g[c * C::n + j - shift]) : 0.f;
      } else {
        C::load(a.g + (int64_t)c * C::n, g);
      }
      float part = 0.f;  // a sum of its own for each chunk keeps the chains of additions short
#pragma unroll
      for (int j = 0; j < C::n; ++j) {
        part = fmaf(s[i][j], s[i][j], part);
        s[i][j] *= g[j];
        top = max_nan(top, fabsf(s[i][j]));
      }
      sum += part;
    }
    team_reduce(sum, top, team / 32, which * (team / 32), red[turn ^= 1]);
    const float inv = 1.f / sqrtf(sum / (float)a.d + a.eps);
    const float scale = row_scale(top, inv), f8 = 1.f / scale;
    if (t < a.N && a.out8 && in_team == 0) a.scale8[t] = scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = in_team + i * team;
      if (c >= chunks) continue;
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
    place(t + step);
  }
}

// Rows too long for one CTA's registers: x and residual are read again (from L2) for the outputs,
// element by element, so each output may only be the input it replaces element for element.
template <typename T>
__global__ void __launch_bounds__(1024) rmsnorm_long_kernel(const NormArgs<T> a) {
  __shared__ float red[2][64];
  int turn = 0;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t = blockIdx.x; t < a.N; t += gridDim.x) {
    const int64_t base = t * a.d;
    float sum = 0.f, top = 0.f;
    for (int64_t c = threadIdx.x; c < a.d; c += blockDim.x) {
      float s = to_float(a.x[base + c]);
      if (a.res) s += to_float(a.res[base + c]);
      sum = fmaf(s, s, sum);
      top = max_nan(top, fabsf(s * to_float(a.g[c])));
    }
    team_reduce(sum, top, blockDim.x / 32, 0, red[turn ^= 1]);
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


// Measured on GB300 (three sets of buffers in turn):
//  - a row costs a fixed time (two barriers, two trips through shared memory) besides its bytes, so many
//    values a thread and few threads a row win: 16 fp32 values (1237 x 2049: 7.0 us, 9.9 with 8);
//  - bf16 loads are in flight half of the time only, which fetching a row ahead fills: 8192 x 4096
//    with a residual and all outputs 48.1 us (6280 GB/s; 32 values a thread) against 54.1, without a
//    residual 27.6 against 29.3, 4096 x 2048 12.2 against 14.6 (16 values, fewer rows an SM: below 16M
//    elements).  In fp32 the registers it takes cost more than it gives (49 against 46 us).
template <typename T, bool kVec, bool kRagged>
cudaError_t launch_norm(const NormArgs<T>& a, cudaStream_t stream) {
  constexpr int n = Chunk<T, kVec>::n;
  constexpr bool may_ahead = n == 8 && !kRagged;
  const int64_t chunks = (a.d + n - 1) / n + (kRagged ? 1 : 0);
  const bool large = a.N * a.d >= (int64_t)16 << 20;
  const bool ahead = may_ahead && a.N >= 8 * num_sms() && chunks <= 4 * 256;
  const int many = n == 1 || n == 4 ? 4 : (ahead ? large || chunks > 512 : kRagged) ? 4 : 2;  // chunks a thread
  int team = 32;
  while (team < 1024 && chunks > (int64_t)team * many) team *= 2;
  while (!ahead && team < 1024 && chunks > team && a.N * team * 2 <= (int64_t)num_sms() * 1024) team *= 2;
  const int per = (int)((chunks + team - 1) / team);
  const int least = n == 8 ? 128 : 256, threads = team < least ? least : team;
  const int64_t groups = (a.N + threads / team - 1) / (threads / team);
  const int64_t most = (int64_t)num_sms() * ((ahead && !(large && a.res) ? 1024 : 2048) / threads);
  const dim3 grid((unsigned)(groups < most ? groups : most)), block(threads);
  if constexpr (may_ahead) {
    if (ahead && per <= 1) return launch_kernel(rmsnorm_kernel<T, kVec, 1, kRagged, true>, grid, block, 0, stream, 0, a, team);
    if (ahead && per <= 2) return launch_kernel(rmsnorm_kernel<T, kVec, 2, kRagged, true>, grid, block, 0, stream, 0, a, team);
    if (ahead) return launch_kernel(rmsnorm_kernel<T, kVec, 4, kRagged, true>, grid, block, 0, stream, 0, a, team);
  }
  if (per <= 1) return launch_kernel(rmsnorm_kernel<T, kVec, 1, kRagged, false>, grid, block, 0, stream, 0, a, team);
  if (per <= 2) return launch_kernel(rmsnorm_kernel<T, kVec, 2, kRagged, false>, grid, block, 0, stream, 0, a, team);
  if (per <= 4) return launch_kernel(rmsnorm_kernel<T, kVec, 4, kRagged, false>, grid, block, 0, stream, 0, a, team);
  if constexpr (n <= 4) {
    if (per <= 8) return launch_kernel(rmsnorm_kernel<T, kVec, 8, kRagged, false>, grid, block, 0, stream, 0, a, team);
  }
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
