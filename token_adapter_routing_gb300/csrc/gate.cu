// gate.cu -- expert-style gate over given logits: softmax or sigmoid scores, a bias that only
// moves the choice, groups of which the best are kept, the k best experts, renormalised weights.
//
// One warp a token; lane l holds the V experts l*V .. l*V+V-1, so among equal values the lowest
// lane, and within it the lowest slot, is the lowest index.
//
// Everything the choice depends on is reproducible: e = expf(l - max) and 1 / (1 + expf(-l)) are
// single fp32 operations, and the softmax's denominator is summed in two fp32 terms (error about
// 2^-46) and rounded once, so it does not depend on the order of the sum.
#include "common.cuh"
#include "kernels.h"

namespace molora {

namespace {

constexpr int kGateWarps = 8;
constexpr uint32_t kFull = 0xffffffffu;
constexpr float kFloatMax = 3.4028234663852886e38f;

// hi + lo += v, without losing v's low bits.  The _rn forms are never fused with the operation
// that made an operand, so every rounding here is the one written.
__device__ __forceinline__ void two_sum(float& hi, float& lo, float v) {
  const float s = __fadd_rn(hi, v), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(v, b)));
  hi = s;
}

// Order-preserving map of a float (not NaN) to an unsigned integer; -inf maps above 0.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);  // -0 and +0 are equal
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

}  // namespace

template <typename T, int V>
__global__ void __launch_bounds__(kGateWarps * 32)
    gate_topk_kernel(const T* __restrict__ logits, int64_t N, int32_t K, bool sigmoid, const float* __restrict__ bias,
                     int32_t G, int32_t keep, int32_t group_top, int32_t k, bool renorm, float scale,
                     int32_t* __restrict__ ids, float* __restrict__ w, int32_t* err_word) {
  extern __shared__ float choice[];  // [warps][K] with groups
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float inf = __int_as_float(0x7f800000);
  const bool by_logit = !bias && (G == 1 || group_top == 1);
  const int a0 = lane * V;
  pdl_wait();
  pdl_launch_dependents();
  float b[V];
#pragma unroll
  for (int i = 0; i < V; ++i) b[i] = bias && a0 + i < K ? bias[a0 + i] : 0.f;
  for (int64_t t = (int64_t)blockIdx.x * kGateWarps + warp; t < N; t += (int64_t)gridDim.x * kGateWarps) {
    float l[V], s[V], c[V];
    bool bad = false;
    float m = -inf;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      l[i] = a0 + i < K ? to_float(logits[t * K + a0 + i]) : -inf;
      bad |= l[i] != l[i] || b[i] != b[i];
      if (l[i] != l[i]) l[i] = -inf;
      l[i] = fminf(l[i], kFloatMax);
      m = fmaxf(m, l[i]);
    }
    if (__any_sync(kFull, bad) && lane == 0) report(err_word, MOLORA_DEV_BAD_LOGIT);
    if (sigmoid) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l[i])));
    } else {
#pragma unroll
      for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
      float hi = 0.f, lo = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = l[i] == -inf ? 0.f : expf(l[i] - m);
        two_sum(hi, lo, s[i]);
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) {
        const float oh = __shfl_xor_sync(kFull, hi, off), ol = __shfl_xor_sync(kFull, lo, off);
        two_sum(hi, lo, oh);
        lo = __fadd_rn(lo, ol);
      }
      const float total = __shfl_sync(kFull, hi + lo, 0);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = total > 0.f ? __fdiv_rn(s[i], total) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      c[i] = l[i] == -inf ? -inf : by_logit ? l[i] : __fadd_rn(s[i], b[i]);
      c[i] = c[i] > -inf ? fminf(c[i], kFloatMax) : -inf;
    }
    if (G > 1) {
      // each group's best, or best two, by 32 / G lanes rounded down to a power of two
      float* mine = choice + (size_t)warp * K;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (a0 + i < K) mine[a0 + i] = c[i];
      __syncwarp();
      const int per = K / G;
      int lanes = 1;
      while (lanes * 2 * G <= 32) lanes *= 2;
      const int g = lane / lanes;
      float c1 = -inf, c2 = -inf;
      if (g < G) {
        for (int i = lane % lanes; i < per; i += lanes) {
          const float v = mine[g * per + i];
          if (v > c1) c2 = c1, c1 = v;
          else if (v > c2) c2 = v;
        }
      }
      for (int off = 1; off < lanes; off <<= 1) {
        const float o1 = __shfl_xor_sync(kFull, c1, off), o2 = __shfl_xor_sync(kFull, c2, off);
        c2 = fmaxf(fminf(c1, o1), fmaxf(c2, o2));
        c1 = fmaxf(c1, o1);
      }
      const float rank = group_top == 1 ? c1 : c1 + c2;
      uint32_t kept = 0;  // bit g: group g stays
      uint32_t key = g < G && lane % lanes == 0 ? ordered(rank) : 0u;
      for (int j = 0; j < keep; ++j) {
        const uint32_t best = __reduce_max_sync(kFull, key);
        const int win = __ffs(__ballot_sync(kFull, key == best)) - 1;
        kept |= 1u << (win / lanes);
        if (lane == win) key = 0u;
      }
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (a0 + i < K && !((kept >> ((a0 + i) / per)) & 1u)) c[i] = -inf;
      __syncwarp();
    }
    // k rounds: the largest remaining choice, ties to the lowest lane and slot
    float sum = 0.f, my_w = 0.f;
    int my_id = -1;
    for (int j = 0; j < k; ++j) {
      float best = -inf, bs = 0.f;
      int slot = 0;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c[i] > best) best = c[i], slot = i, bs = s[i];
      const uint32_t key = ordered(best), top = __reduce_max_sync(kFull, key);
      const int win = __ffs(__ballot_sync(kFull, key == top)) - 1;
      const float wv = __shfl_sync(kFull, bs, win), cv = __shfl_sync(kFull, best, win);
      const int id = __shfl_sync(kFull, a0 + slot, win);
      const bool none = cv == -inf;
      if (lane == win)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i == slot) c[i] = -inf;
      if (!none) sum += wv;
      if (lane == j) my_id = none ? -1 : id, my_w = none ? 0.f : wv;
    }
    if (lane < k) {
      if (renorm) my_w = sum > 0.f ? my_w / sum : 0.f;
      ids[t * k + lane] = my_id;
      w[t * k + lane] = my_w * scale;
    }
  }
}

namespace {

template <typename T>
cudaError_t launch_gate_typed(const T* logits, int64_t N, int32_t K, bool sigmoid, const float* bias, int32_t G,
                              int32_t keep, int32_t group_top, int32_t k, bool renorm, float scale, int32_t* ids,
                              float* w, int32_t* err_word, cudaStream_t stream) {
  const int64_t blocks = (N + kGateWarps - 1) / kGateWarps, most = (int64_t)num_sms() * 8;
  const dim3 grid((unsigned)(blocks < most ? blocks : most)), block(kGateWarps * 32);
  const size_t smem = G > 1 ? sizeof(float) * kGateWarps * K : 0;
#define MOLORA_GATE(V)                                                                                              \
  return launch_kernel(gate_topk_kernel<T, V>, grid, block, smem, stream, 0, logits, N, K, sigmoid, bias, G, keep, \
                       group_top, k, renorm, scale, ids, w, err_word)
  if (K <= 32) MOLORA_GATE(1);
  if (K <= 64) MOLORA_GATE(2);
  if (K <= 128) MOLORA_GATE(4);
  if (K <= 256) MOLORA_GATE(8);
  MOLORA_GATE(16);
#undef MOLORA_GATE
}

}  // namespace

cudaError_t launch_gate_topk(const void* logits, molora_dtype dtype, int64_t N, int32_t K, bool sigmoid,
                             const float* bias, int32_t groups, int32_t keep, int32_t group_top, int32_t k, bool renorm,
                             float scale, int32_t* ids, float* w, int32_t* err_word, cudaStream_t stream) {
  if (dtype == MOLORA_BF16)
    return launch_gate_typed(static_cast<const __nv_bfloat16*>(logits), N, K, sigmoid, bias, groups, keep, group_top, k,
                             renorm, scale, ids, w, err_word, stream);
  return launch_gate_typed(static_cast<const float*>(logits), N, K, sigmoid, bias, groups, keep, group_top, k, renorm,
                           scale, ids, w, err_word, stream);
}

}  // namespace molora
