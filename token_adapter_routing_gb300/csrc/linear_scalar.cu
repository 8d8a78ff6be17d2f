// linear_scalar.cu -- the base product with its epilogue on CUDA cores, for every type, size and
// alignment:
//
//   y[t,o] = act(sx[t] * sw[o] * sum_i x[t,i] W[o,i] + bias[o]) + residual[t,o]
//
// A CTA of 256 threads makes a 64 x 64 tile of y; each thread 4 x 4 of it, by fp32 FMAs over
// K steps of 16 that are converted to fp32 on their way into shared memory.
#include "common.cuh"
#include "kernels.h"
#include "linear.cuh"

namespace molora {

namespace {

constexpr int kTile = 64, kStep = 16, kPad = 4;

}  // namespace

template <typename T, typename Y>
__global__ void __launch_bounds__(256)
    linear_scalar_kernel(const T* __restrict__ x, const float* __restrict__ sx, int64_t N, int32_t d_in,
                         const T* __restrict__ W, const float* __restrict__ sw, int32_t d_out,
                         const float* __restrict__ bias, molora_activation act, const Y* residual, Y* y) {
  __shared__ float xs[kStep][kTile + kPad], ws[kStep][kTile + kPad];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const unsigned across = (unsigned)((d_out + kTile - 1) / kTile);
  const int64_t t0 = (int64_t)(blockIdx.x / across) * kTile;
  const int o0 = (int)(blockIdx.x % across) * kTile;
  pdl_wait();
  pdl_launch_dependents();
  float acc[4][4] = {};
  for (int i0 = 0; i0 < d_in; i0 += kStep) {
    // thread: column i0 + tx of rows ty, ty + 16, ...
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = ty + 16 * r, i = i0 + tx;
      xs[tx][row] = i < d_in && t0 + row < N ? to_float(x[(t0 + row) * d_in + i]) : 0.f;
      ws[tx][row] = i < d_in && o0 + row < d_out ? to_float(W[(int64_t)(o0 + row) * d_in + i]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kStep; ++kk) {
      const float4 a = *reinterpret_cast<const float4*>(&xs[kk][ty * 4]);
      const float4 b = *reinterpret_cast<const float4*>(&ws[kk][tx * 4]);
      const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] = fmaf(av[p], bv[q], acc[p][q]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int64_t t = t0 + ty * 4 + p;
    if (t >= N) continue;
    const float st = sx ? sx[t] : 1.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int o = o0 + tx * 4 + q;
      if (o >= d_out) continue;
      float v = acc[p][q] * st;
      if (sw) v *= sw[o];
      if (bias) v += bias[o];
      v = activate(v, act);
      if (residual) v += to_float(residual[t * d_out + o]);
      store_as(y + t * d_out + o, v);
    }
  }
}

namespace {

template <typename T, typename Y>
cudaError_t launch_scalar(const LinearArgs& a, cudaStream_t stream) {
  const dim3 grid((unsigned)(((a.N + kTile - 1) / kTile) * ((a.d_out + kTile - 1) / kTile)));
  return launch_kernel(linear_scalar_kernel<T, Y>, grid, dim3(256), 0, stream, 0, static_cast<const T*>(a.x), a.x_scale,
                       a.N, a.d_in, static_cast<const T*>(a.W), a.w_scale, a.d_out, a.bias, a.act,
                       static_cast<const Y*>(a.residual), static_cast<Y*>(a.y));
}

template <typename T>
cudaError_t launch_scalar_y(const LinearArgs& a, cudaStream_t stream) {
  return a.y_bf16 ? launch_scalar<T, __nv_bfloat16>(a, stream) : launch_scalar<T, float>(a, stream);
}

}  // namespace

cudaError_t launch_linear_scalar(const LinearArgs& a, cudaStream_t stream) {
  if (a.dtype == MOLORA_BF16) return launch_scalar_y<__nv_bfloat16>(a, stream);
  if (a.dtype == MOLORA_E4M3) return launch_scalar_y<__nv_fp8_e4m3>(a, stream);
  return launch_scalar_y<float>(a, stream);
}

}  // namespace molora
